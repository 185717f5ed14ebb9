"""Refusals of the paged cache's entry points that need no GPU: every argument is checked before a
device is touched (the pointer values below are never dereferenced)."""
import ctypes

import pytest
import torch

import invariant_deterministic_gemm_bi_b200 as bg
from invariant_deterministic_gemm_bi_b200 import binding

S = binding.STATUS
BAD, ALIGN, SHAPE = S["BI_ERR_INVALID_ARG"], S["BI_ERR_ALIGNMENT"], S["BI_ERR_UNSUPPORTED_SHAPE"]
FINE = {0, S["BI_ERR_NO_DEVICE"]}   # accepted arguments, on a machine without a GPU


def cache(**change):
    a = dict(k=256, v=256, k_scale=256, v_scale=256, num_pages=10, page_size=16, num_heads=2, head_dim=128,
             page_stride=16 * 256, token_stride=256, head_stride=128) | change
    return ctypes.pointer(binding.KvCacheView(*a.values()))


CACHES = [({"k": None}, BAD), ({"v": None}, BAD), ({"k_scale": None}, BAD), ({"v_scale": None}, BAD),
          ({"num_pages": 0}, BAD), ({"num_heads": 0}, BAD), ({"page_size": 0}, SHAPE), ({"page_size": 24}, SHAPE),
          ({"page_size": 512}, SHAPE), ({"head_dim": 96}, SHAPE), ({"head_dim": 256}, SHAPE),
          ({"num_pages": 2 ** 27}, SHAPE), ({"token_stride": 112}, BAD), ({"head_stride": 64}, BAD),
          ({"page_stride": 15 * 256}, BAD), ({"page_stride": -4096}, BAD), ({"token_stride": 2 ** 62}, SHAPE),
          ({"head_stride": 2 ** 62}, SHAPE), ({"page_stride": 2 ** 62}, SHAPE), ({"k": 264}, ALIGN), ({"v": 8}, ALIGN),
          ({"k_scale": 258}, ALIGN), ({"page_stride": 4104}, ALIGN), ({"token_stride": 264, "page_stride": 8192}, ALIGN),
          ({"head_stride": 256, "token_stride": 128, "page_stride": 8192}, BAD), ({"token_stride": 128}, BAD),
          ({"head_stride": 136, "token_stride": 272, "page_stride": 8192}, ALIGN)]


@pytest.mark.parametrize("change,status", CACHES)
def test_cache_handles(change, status):
    lib = binding.load_library()
    c = cache(**change)
    assert lib.bi_kv_append_e4m3(c, 256, 256, 256, 256, 256, 1, None) == status
    assert lib.bi_paged_decode_attention(c, 256, 1024, 256, 4, 4, 256, 1, 8, 0.1, 0, None, 0, 256, 1024, None, None) == status


def test_no_cache_handle():
    lib = binding.load_library()
    assert lib.bi_kv_append_e4m3(None, 256, 256, 256, 256, 256, 1, None) == BAD
    assert lib.bi_paged_decode_attention(None, 256, 1024, 256, 4, 4, 256, 1, 8, 0.1, 0, None, 0, 256, 1024, None, None) == BAD


@pytest.mark.parametrize("change,status", [
    ({"T": -1}, BAD), ({"ldk": 248}, BAD), ({"ldv": 0}, BAD), ({"K": None}, BAD), ({"V": None}, BAD), ({"slots": None}, BAD),
    ({"K": 264}, ALIGN), ({"V": 2}, ALIGN), ({"ldk": 260}, ALIGN), ({"ldv": 257}, ALIGN), ({"slots": 258}, ALIGN),
    ({"T": 2 ** 31}, SHAPE), ({"ldk": 2 ** 40}, SHAPE), ({"T": 0, "K": None, "slots": None}, 0)])
def test_append(change, status):
    a = dict(K=256, ldk=256, V=256, ldv=256, slots=256, T=3) | change
    assert binding.load_library().bi_kv_append_e4m3(cache(), *a.values(), None) == status


@pytest.mark.parametrize("change,status", [
    ({"B": -1}, BAD), ({"max_pages": -1}, BAD), ({"ld_table": 3}, BAD), ({"max_tokens": -1}, BAD), ({"capacity": -1}, BAD),
    ({"page": 0}, SHAPE), ({"page": 48}, SHAPE), ({"B": 8193}, SHAPE), ({"max_pages": 2 ** 28, "ld_table": 2 ** 28}, SHAPE),
    ({"max_tokens": 2 ** 31}, SHAPE), ({"capacity": 2 ** 31}, SHAPE), ({"ctx": None}, BAD), ({"new": None}, BAD),
    ({"stack": None}, BAD), ({"count": None}, BAD), ({"table": None}, BAD), ({"lens": None}, BAD), ({"offsets": None}, BAD),
    ({"slots": None}, BAD), ({"left": None}, BAD), ({"status": None}, BAD), ({"ctx": 257}, ALIGN), ({"new": 258}, ALIGN),
    ({"table": 259}, ALIGN), ({"slots": 257}, ALIGN), ({"positions": 257}, ALIGN), ({"status": 2}, ALIGN)])
def test_block_tables(change, status):
    a = dict(ctx=256, new=256, B=2, page=16, stack=256, capacity=8, count=256, table=256, ld_table=4, max_pages=4, lens=256,
             offsets=256, slots=256, positions=None, max_tokens=4, left=256, status=256) | change
    assert binding.load_library().bi_kv_block_tables(*a.values(), None) == status


@pytest.mark.parametrize("change,status", [
    ({"B": -1}, BAD), ({"Hq": 0}, BAD), ({"max_pages": -1}, BAD), ({"ld_table": 3}, BAD), ({"window": -1}, BAD),
    ({"ldq": 1016}, BAD), ({"ldo": 8}, BAD), ({"scale": float("nan")}, BAD), ({"scale": float("inf")}, BAD),
    ({"Hq": 7, "ldq": 4096}, SHAPE), ({"Hq": 34, "ldq": 8192, "ldo": 8192}, SHAPE), ({"max_pages": 2 ** 27, "ld_table": 2 ** 27}, SHAPE),
    ({"B": 2 ** 31}, SHAPE), ({"B": 16385}, SHAPE), ({"max_pages": 2 ** 26 + 1, "ld_table": 2 ** 27}, SHAPE), ({"ldq": 2 ** 60}, SHAPE), ({"Q": None}, BAD), ({"table": None}, BAD), ({"lens": None}, BAD),
    ({"O": None}, BAD), ({"Q": 264}, ALIGN), ({"O": 264}, ALIGN), ({"ldq": 1028}, ALIGN), ({"ldo": 1028}, ALIGN),
    ({"table": 258}, ALIGN), ({"lens": 257}, ALIGN), ({"lse": 258}, ALIGN), ({"B": 0, "Q": None, "O": None}, 0)])
def test_attention(change, status):
    a = dict(Q=256, ldq=1024, table=256, ld_table=4, max_pages=4, lens=256, B=2, Hq=8, scale=0.1, window=0, ws=None,
             ws_bytes=0, O=256, ldo=1024, lse=None) | change
    assert binding.load_library().bi_paged_decode_attention(cache(), *a.values(), None) == status


def test_attention_checks_its_workspace():
    run = binding.load_library().bi_paged_decode_attention
    pages = 4096
    need = bg.bi_paged_decode_attention_workspace_bytes(2, 8, 128, pages * 16)
    args = lambda ws, n: (cache(), 256, 1024, 256, pages, pages, 256, 2, 8, 0.1, 0, ws, n, 256, 1024, None, None)
    if need:
        assert run(*args(None, need)) == BAD and run(*args(256, need - 1)) == BAD and run(*args(264, need)) == ALIGN
    for sizes in ((0, 8, 128, 1000), (2, 0, 128, 1000), (2, 8, 0, 1000), (2, 8, 128, 0), (-1, 8, 128, 99999)):
        assert bg.bi_paged_decode_attention_workspace_bytes(*sizes) == 0


@pytest.mark.parametrize("sizes", [(1, 8, 128, 2 ** 30 + 1), (1, 8, 128, 2 ** 38 + 1), (1, 8, 64, 2 ** 39 + 1),
                                   (1, 8, 128, 2 ** 62), (1, 8, 128, 2 ** 63 - 1), (16385, 8, 128, 4096),
                                   (2 ** 62, 8, 128, 4096), (16384, 2 ** 17, 128, 4096), (1, 8, 96, 4096),
                                   (1, 8, 2 ** 31 - 1, 4096)])
def test_workspace_sizes_beyond_the_limits_are_zero(sizes):
    # max_len from 2^38 on once did not return, from 2^30 on the number was of a truncated length
    assert bg.bi_paged_decode_attention_workspace_bytes(*sizes) == 0


def test_the_largest_workspace_sizes():
    assert bg.bi_paged_decode_attention_workspace_bytes(1, 8, 128, 2 ** 30) == 8 * 128 * 130 * 4
    assert bg.bi_paged_decode_attention_workspace_bytes(16384, 2 ** 17 - 1, 64, 2 ** 30) == 16384 * (2 ** 17 - 1) * 128 * 66 * 4


def test_accepted_arguments_reach_the_device_probe():
    if torch.cuda.is_available():
        pytest.skip("the pointers are made up")
    lib = binding.load_library()
    assert lib.bi_kv_append_e4m3(cache(), 256, 256, 256, 256, 256, 3, None) in FINE
    assert lib.bi_kv_block_tables(256, 256, 2, 16, 256, 8, 256, 256, 4, 4, 256, 256, 256, None, 4, 256, 256, None) in FINE
    assert lib.bi_paged_decode_attention(cache(), 256, 1024, 256, 4, 4, 256, 1, 8, 0.1, 0, None, 0, 256, 1024, None, None) in FINE


def test_the_binding_refuses_what_the_abi_cannot_see():
    k = torch.zeros((3, 16, 2, 64), dtype=torch.uint8)
    s = torch.ones((3, 2))
    bg.KvCache(k, k.clone(), s, s.clone())
    for bad in (lambda: bg.KvCache(k.float(), k, s, s), lambda: bg.KvCache(k, k[:2], s, s),
                lambda: bg.KvCache(k, k.transpose(1, 2).contiguous().transpose(1, 2), s, s),
                lambda: bg.KvCache(k[..., ::2], k[..., ::2], s, s), lambda: bg.KvCache(k, k, s[:2], s),
                lambda: bg.KvCache(k, k, s.double(), s), lambda: bg.KvCache(k[0], k[0], s, s)):
        with pytest.raises((TypeError, ValueError)):
            bad()
    c = bg.KvCache(k, k.clone(), s, s.clone())
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    i4 = torch.zeros(4, dtype=torch.int32)
    for K, V, slots in ((x.float(), x, i4), (x, x[:3], i4), (x, x, i4.long()), (x, x, i4[:3]), (x[:, :1], x, i4),
                        (x, x.transpose(0, 1).contiguous().transpose(0, 1), i4), (x, x, i4.repeat(2)[::2])):
        with pytest.raises((TypeError, ValueError)):
            bg.bi_kv_append_e4m3(c, K, V, slots)
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    t, n = torch.zeros((2, 3), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for Q, T, L, O, lse in ((q.float(), t, n, q, None), (q, t.long(), n, q, None), (q, t[:1], n, q, None),
                            (q, t, n[:1], q, None), (q, t, n, q[:1], None), (q, t, n, q.float(), None),
                            (q, t, n, q, torch.zeros((2, 3))), (q, t.repeat(1, 2)[:, ::2], n, q, None),
                            (torch.zeros((2, 4, 128), dtype=torch.bfloat16), t, n, q, None)):
        with pytest.raises((TypeError, ValueError)):
            bg.bi_paged_decode_attention(c, Q, T, L, O, 0.1, lse=lse)
    one = torch.zeros(1, dtype=torch.int32)
    three = torch.zeros(3, dtype=torch.int32)
    good = dict(ctx_lens=n, new_lens=n.clone(), page_size=16, free_pages=i4, free_count=one, block_table=t, seq_lens=n.clone(),
                token_offsets=three, slot_map=i4.clone(), free_left=one.clone(), status=one.clone())
    for change in ({"ctx_lens": n.long()}, {"new_lens": one}, {"seq_lens": three}, {"token_offsets": n}, {"block_table": t[:1]},
                   {"free_count": n}, {"free_left": n}, {"status": n}, {"positions": one}, {"slot_map": i4.float()}):
        with pytest.raises((TypeError, ValueError)):
            bg.bi_kv_block_tables(**(good | change))


@pytest.mark.parametrize("shape", [(64,), (2, 256), (1, 2, 4, 64), ()])
def test_queries_of_other_shapes_are_refused(shape):
    k, s = torch.zeros((3, 16, 2, 64), dtype=torch.uint8), torch.ones((3, 2))
    c = bg.KvCache(k, k.clone(), s, s.clone())
    Q = torch.zeros(shape, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        bg.bi_paged_decode_attention(c, Q, torch.zeros((2, 3), dtype=torch.int32), torch.zeros(2, dtype=torch.int32), Q, 0.1)
