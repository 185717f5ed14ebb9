"""The current stream's handle in the binding, with and without torch's private way to it (no GPU)."""
from types import SimpleNamespace

import pytest
import torch

from invariant_deterministic_gemm_bi_b200 import binding


@pytest.fixture
def fake_cuda(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: SimpleNamespace(cuda_stream=1000 + device))
    return monkeypatch


def test_the_private_call_is_used_where_torch_has_it(fake_cuda):
    fake_cuda.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 50 + device, raising=False)
    assert binding._stream_handle(None) == 53 and binding._stream_on(torch, 2, None) == 52


def test_the_public_call_serves_where_it_has_not(fake_cuda):
    fake_cuda.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    assert binding._stream_handle(None) == 1003 and binding._stream_on(torch, 2, None) == 1002


def test_given_streams_and_no_device():
    assert binding._stream_handle(7) == 7 and binding._stream_handle(SimpleNamespace(cuda_stream=9)) == 9
    assert binding._stream_on(torch, 0, 7) == 7 and binding._stream_on(torch, -1, None) is None
