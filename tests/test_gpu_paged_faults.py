"""Waits of the paged decode attention that run out, without a GPU fault.

A test-only switch makes every thread block's producer leave one load out, so a wait for it can never
complete and ends by its limit of 20 ms.  What the block has finished by then is right, the rest of
its outputs is NaN and nothing is left as it was; the next call is right."""
import pytest
import torch

import invariant_deterministic_gemm_bi_b200 as bg
from tests.kv_util import DEV, Paged, attend, queries

pytestmark = pytest.mark.gpu


def check(P, table, lens, Q, n, scale=0.1):
    """(outputs missing, outputs there) of a call whose blocks leave their n-th load out."""
    want, wlse = attend(P.cache, Q, table, lens, scale)
    assert not torch.isnan(want.float()).any()
    guard = torch.full((Q.shape[0] + 2, *Q.shape[1:]), 3.0, dtype=torch.bfloat16, device=DEV)
    bg.bi_paged_decode_attention_set_wait_timeout(20_000_000)
    bg.bi_paged_decode_attention_debug_skip_load(n)
    try:
        O, lse = attend(P.cache, Q, table, lens, scale, out=guard[1:-1])
    finally:
        bg.bi_paged_decode_attention_debug_skip_load(0)
        bg.bi_paged_decode_attention_set_wait_timeout(0)
    missing = torch.isnan(O.float())
    assert torch.all(missing | (O.view(torch.int16) == want.view(torch.int16)))
    assert torch.all(torch.isnan(lse) | (lse == wlse))
    assert torch.all(guard[0] == 3) and torch.all(guard[-1] == 3)
    empty = lens == 0
    assert not missing[empty].any() and torch.isneginf(lse[empty]).all()
    again, alse = attend(P.cache, Q, table, lens, scale)
    assert torch.equal(again.view(torch.int16), want.view(torch.int16)) and torch.equal(alse, wlse)
    return missing[~empty], lse[~empty]


@pytest.mark.parametrize("Hq,heads,D", [(8, 2, 128), (16, 2, 128), (32, 2, 128), (8, 2, 64), (32, 2, 64)])
@pytest.mark.parametrize("page", [16, 64])
def test_a_first_load_that_never_comes(Hq, heads, D, page):
    P = Paged([100, 0, 700, 1, 3000, 260], heads, D, page, seed=40)
    missing, lse = check(P, P.dtable, P.dlens, queries(6, Hq, D, 41), 1)
    assert missing.all() and torch.isnan(lse).all()


@pytest.mark.parametrize("Hq,heads,D", [(8, 8, 64), (64, 8, 128), (32, 2, 128)])
@pytest.mark.parametrize("n", [2, 3, 10, 67, 300, 301])
def test_a_later_load_that_never_comes(Hq, heads, D, n):
    # up to two hundred items a block, so that tables of items have been refilled by the time of the last ones
    B = 2000 if heads == 8 else 4000
    P = Paged([300, 290], heads, D, 64, seed=42)
    row = torch.arange(B, device=DEV) % 2
    lens = P.dlens[row].contiguous()
    lens[77] = 0
    missing, lse = check(P, P.dtable[row].contiguous(), lens, queries(2, Hq, D, 43)[row].contiguous(), n)
    # two chunks of one step a sequence and head, two loads each, dealt evenly to the blocks
    blocks = torch.cuda.get_device_properties(0).multi_processor_count
    loads = 4 * (B - 1) * heads // blocks
    share = missing.float().mean().item()
    if n <= loads:
        assert share >= 1 - (n + 2) / loads and (n < 67 or share < 1 - n / loads / 3)
    elif n > loads + 2:   # nothing was left out (the two loads behind a block's last only say so)
        assert share == 0 and not torch.isnan(lse).any()


def test_long_sequences_whose_last_load_never_comes():
    # chunks of four steps: blocks that give up late leave parts of sequences whose other parts are there
    P = Paged([30000, 9000], 2, 128, 64, seed=44)
    missing, lse = check(P, P.dtable, P.dlens, queries(2, 16, 128, 45), 8)
    assert missing.any()


def test_a_limit_that_is_long_enough_changes_nothing():
    P = Paged([3000, 40], 2, 128, 32, seed=46)
    Q = queries(2, 16, 128, 47)
    want, wlse = attend(P.cache, Q, P.dtable, P.dlens, 0.1)
    for ns in (200_000_000, 2 ** 64 - 1, 0):
        bg.bi_paged_decode_attention_set_wait_timeout(ns)
        O, lse = attend(P.cache, Q, P.dtable, P.dlens, 0.1)
        assert torch.equal(O.view(torch.int16), want.view(torch.int16)) and torch.equal(lse, wlse)
