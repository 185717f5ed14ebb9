"""Decode attention over the paged 8-bit cache on the GPU, against the fp64 oracle and bitwise
against itself in other batches, page sizes and layouts."""
import numpy as np
import pytest
import torch

import invariant_deterministic_gemm_bi_b200 as bg
from invariant_deterministic_gemm_bi_b200 import inputs
from oracle import kv_cache as okv
from tests.kv_util import DEV, NAN_CODE, Paged, assert_attention, attend, pool, queries, softmax_scale

pytestmark = pytest.mark.gpu
EDGES = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 511, 512, 513]


def check(P, Hq, heads, D, seed, window=0, std=1.0, scale=None):
    Q = queries(len(P.lens), Hq, D, seed, std)
    scale = softmax_scale(D) if scale is None else scale
    O, lse = attend(P.cache, Q, P.dtable, P.dlens, scale, window)
    K, V = P.values()
    ref = okv.paged_attention(inputs.to_numpy_bits(Q), K, V, P.table, P.lens, scale, window,
                              P.v_scale.cpu().numpy())
    assert_attention(O, lse, ref, scale, D)
    return Q, O, lse


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("D", [64, 128])
def test_every_length_edge(page, D):
    check(Paged(EDGES, 2, D, page, seed=100 + page + D), 8, 2, D, seed=1)


@pytest.mark.parametrize("Hq,heads", [(1, 1), (3, 3), (5, 1), (14, 2), (16, 2), (9, 1), (12, 1), (32, 2), (48, 3)])
@pytest.mark.parametrize("D", [64, 128])
def test_head_layouts(Hq, heads, D):
    check(Paged([1, 77, 600, 0, 1300], heads, D, 32, seed=200 + Hq), Hq, heads, D, seed=2)


@pytest.mark.parametrize("lens", [[2049, 4095, 4096, 4097], [8191, 8192, 8193], [16384, 16385, 1], [40001], [70000, 3]])
def test_long_sequences(lens):
    check(Paged(lens, 1, 128, 64, seed=300 + lens[0]), 4, 1, 128, seed=3)


@pytest.mark.parametrize("Hq,heads,D", [(16, 4, 128), (32, 4, 128), (32, 2, 128), (32, 4, 64), (32, 2, 64)])
def test_long_chunks_of_many_heads(Hq, heads, D):
    # chunks of several steps, more of them than CTAs, so that a CTA's two halves drift apart
    check(Paged([30001, 20000, 70], heads, D, 128, seed=350 + Hq + D), Hq, heads, D, seed=3)


@pytest.mark.parametrize("window", [1, 16, 17, 100, 256, 1000, 1 << 40])
def test_windows(window):
    P = Paged([0, 1, 16, 17, 99, 100, 101, 255, 256, 257, 1000, 1001, 1500], 2, 128, 16, seed=400)
    # pages wholly before the window are never looked up: their table entries may be anything
    for b, n in enumerate(P.lens):
        P.table[b, :max(0, n - window) // 16] = -1
    P.dtable = torch.from_numpy(P.table).to(DEV)
    check(P, 8, 2, 128, seed=4, window=window)


@pytest.mark.parametrize("layout", ["head", "wide"])
def test_layouts_give_the_same_bits(layout):
    lens = [1, 40, 333, 1025]
    a = Paged(lens, 3, 64, 32, seed=500)
    b = Paged(lens, 3, 64, 32, seed=500, layout=layout)
    Q = queries(4, 12, 64, 5)
    Oa, la = attend(a.cache, Q, a.dtable, a.dlens, 0.125)
    Ob, lb = attend(b.cache, Q, b.dtable, b.dlens, 0.125)
    assert torch.equal(Oa.view(torch.int16), Ob.view(torch.int16)) and torch.equal(la, lb)


@pytest.mark.parametrize("std,scale", [(1.0, 1e-30), (1.0, 0.0), (30.0, 0.25), (1e-30, 1.0), (1e30, 1e-31), (1.0, -0.5)])
def test_flat_sharp_tiny_and_huge_scores(std, scale):
    check(Paged([5, 300, 2000], 2, 128, 64, seed=600), 8, 2, 128, seed=6, std=std, scale=scale)


def test_queries_of_mixed_magnitudes():
    P = Paged([700, 40], 1, 128, 64, seed=620)
    Q = queries(2, 4, 128, 7) * torch.exp2(torch.randint(-60, 20, (2, 4, 128), device=DEV).float()).to(torch.bfloat16)
    O, lse = attend(P.cache, Q, P.dtable, P.dlens, 2.0 ** -16)
    K, V = P.values()
    ref = okv.paged_attention(inputs.to_numpy_bits(Q), K, V, P.table, P.lens, 2.0 ** -16,
                              v_scale=P.v_scale.cpu().numpy())
    assert_attention(O, lse, ref, 2.0 ** -16, 128)


def test_value_scales_far_apart_and_zero_blocks():
    # the value scales of neighbouring pages differ by up to 2^40; two pages are all zeros with the
    # smallest scale, as the write leaves them
    P = Paged([200, 1000], 1, 128, 16, seed=630, scales="one")
    s = 2.0 ** torch.randint(-20, 21, (P.pages, 1), device=DEV).float()
    P.v_scale.copy_(s)
    for p in (int(P.table[1, 3]), int(P.table[1, 30])):
        P.v[p].zero_()
        P.v_scale[p] = 2.0 ** -64
    check(P, 4, 1, 128, seed=8)
    P.v_scale.fill_(2.0 ** -64)
    check(P, 4, 1, 128, seed=8)
    P.v_scale.fill_(2.0 ** 64)
    check(P, 4, 1, 128, seed=8)


def test_a_sequence_does_not_see_its_batch():
    lens = [1200, 17, 0, 256, 513, 3000, 64, 900, 31, 2048]
    P = Paged(lens, 2, 128, 32, seed=700)
    Q = queries(len(lens), 16, 128, 9)
    O, lse = attend(P.cache, Q, P.dtable, P.dlens, 0.1)
    for b in range(len(lens)):
        Ob, lb = attend(P.cache, Q[b:b + 1], P.dtable[b:b + 1], P.dlens[b:b + 1], 0.1)
        assert torch.equal(Ob.view(torch.int16)[0], O.view(torch.int16)[b]) and torch.equal(lb[0], lse[b])
    perm = torch.randperm(len(lens), device=DEV)
    Op, lp = attend(P.cache, Q[perm], P.dtable[perm], P.dlens[perm].contiguous(), 0.1)
    assert torch.equal(Op.view(torch.int16), O.view(torch.int16)[perm]) and torch.equal(lp, lse[perm])
    # a wider table (a larger workspace and another grid) changes nothing either
    wide = torch.full((len(lens), 700), -1, dtype=torch.int32, device=DEV)
    wide[:, :P.width] = P.dtable
    Ow, lw = attend(P.cache, Q, wide, P.dlens, 0.1)
    assert torch.equal(Ow.view(torch.int16), O.view(torch.int16)) and torch.equal(lw, lse)


def test_page_numbers_and_page_size_do_not_matter():
    n, heads, D = 1111, 2, 128
    small = Paged([n], heads, D, 16, seed=800, scales="one")
    Q = queries(1, 8, D, 10)
    O, lse = attend(small.cache, Q, small.dtable, small.dlens, 0.09)
    for page in (32, 64, 128, 256):
        k, v = pool(90, page, heads, D), pool(90, page, heads, D)
        order = torch.randperm(90, device=DEV)[:-(-n // page)]
        rows = torch.arange(n, device=DEV)
        src = small.dtable[0].long()
        at = order[rows // page]
        k[at, rows % page] = small.k[src[rows // 16], rows % 16]
        v[at, rows % page] = small.v[src[rows // 16], rows % 16]
        one = torch.ones((90, heads), device=DEV)
        table = order.to(torch.int32)[None].contiguous()
        Op, lp = attend(bg.KvCache(k, v, one, one.clone()), Q, table, small.dlens, 0.09)
        assert torch.equal(Op.view(torch.int16), O.view(torch.int16)) and torch.equal(lp, lse), page


def test_query_tokens_of_one_sequence_as_rows():
    # four draft tokens: rows that share the sequence's pages, each with its own length
    P = Paged([401], 2, 128, 64, seed=820)
    Q = queries(4, 8, 128, 11)
    table, lens = P.dtable.expand(4, -1).contiguous(), torch.tensor([398, 399, 400, 401], dtype=torch.int32, device=DEV)
    O, lse = attend(P.cache, Q, table, lens, 0.1)
    for i in range(4):
        Oi, li = attend(P.cache, Q[i:i + 1], P.dtable, lens[i:i + 1], 0.1)
        assert torch.equal(Oi.view(torch.int16)[0], O.view(torch.int16)[i]) and torch.equal(li[0], lse[i])


def test_bad_lengths_pages_and_scales_give_nan_to_their_rows_only():
    lens = [100, 700, 40, 300, 520, 90]
    P = Paged(lens, 2, 128, 16, seed=900, scales="pow2")
    Q = queries(6, 8, 128, 12)
    good, glse = attend(P.cache, Q, P.dtable, P.dlens, 0.1)
    lens_bad = P.dlens.clone()
    lens_bad[0], lens_bad[2] = -1, P.width * 16 + 1
    table = P.dtable.clone()
    table[1, 43] = P.pages          # the last page of row 1
    table[3, 0] = -1
    P.k_scale[P.table[4, 3], 1] = float("nan")
    P.v_scale[P.table[5, 2], 0] = 0.0
    O, lse = attend(P.cache, Q, table, lens_bad, 0.1)
    nan = torch.isnan(O.float()).all(-1)
    want = torch.zeros((6, 8), dtype=torch.bool, device=DEV)
    want[[0, 1, 2, 3]] = True
    want[4, 4:], want[5, :4] = True, True
    assert torch.equal(nan, want) and torch.equal(torch.isnan(lse), want)
    assert torch.equal(O.view(torch.int16)[~want], good.view(torch.int16)[~want]) and torch.equal(lse[~want], glse[~want])


def test_nan_codes_reach_their_head_only():
    P = Paged([300, 80], 2, 64, 64, seed=910)
    Q = queries(2, 8, 64, 13)
    good, glse = attend(P.cache, Q, P.dtable, P.dlens, 0.125)
    P.k[P.table[0, 2], 5, 1, 7] = NAN_CODE            # a key: every output of its heads
    P.v[P.table[1, 0], 3, 0, 9] = NAN_CODE            # a value: its dimension
    O, lse = attend(P.cache, Q, P.dtable, P.dlens, 0.125)
    want = torch.zeros((2, 8, 64), dtype=torch.bool, device=DEV)
    want[0, 4:], want[1, :4, 9] = True, True
    assert torch.equal(torch.isnan(O.float()), want)
    assert torch.equal(O.view(torch.int16)[~want], good.view(torch.int16)[~want])
    assert torch.isnan(lse[0, 4:]).all() and torch.equal(lse[0, :4], glse[0, :4]) and torch.equal(lse[1], glse[1])


def test_slices_of_wider_rows_and_guard_rows():
    # Q is a slice of a projection's output; O has a pitch and rows around it that stay as they were
    P = Paged([50, 0, 513], 2, 128, 64, seed=920)
    wide = inputs.bf16_gaussian((3, 8 * 128 + 520), seed=14, device=DEV)
    Q = wide[:, 256:256 + 1024].view(3, 8, 128)
    buf = torch.full((7, 8 * 128 + 64), 3.0, dtype=torch.bfloat16, device=DEV)
    O = buf[2:5, :1024].view(3, 8, 128)
    attend(P.cache, Q, P.dtable, P.dlens, 0.1, out=O, lse=False)
    want, _ = attend(P.cache, Q.contiguous(), P.dtable, P.dlens, 0.1)
    assert torch.equal(O.view(torch.int16), want.view(torch.int16)) and torch.all(O[1] == 0)
    assert torch.all(buf[:2] == 3) and torch.all(buf[5:] == 3) and torch.all(buf[2:5, 1024:] == 3)


def test_offsets_beyond_32_bits():
    # 4.5 GiB of codes per pool: the last page's offset needs 33 bits
    page, heads, D = 64, 1, 128
    pages = (9 << 29) // (page * heads * D)
    k = torch.zeros((pages, page, heads, D), dtype=torch.uint8, device=DEV)
    v = torch.zeros((pages, page, heads, D), dtype=torch.uint8, device=DEV)
    one = torch.ones((pages, heads), device=DEV)
    small = Paged([130], heads, D, page, seed=930, scales="one")
    at = torch.tensor([pages - 1, 3, pages - 2], device=DEV)
    src = small.dtable[0, :3].long()
    k[at], v[at] = small.k[src], small.v[src]
    Q = queries(1, 4, D, 15)
    O, _ = attend(bg.KvCache(k, v, one, one), Q, at.to(torch.int32)[None].contiguous(), small.dlens, 0.1)
    want, _ = attend(small.cache, Q, small.dtable, small.dlens, 0.1)
    assert torch.equal(O.view(torch.int16), want.view(torch.int16))


def test_a_captured_step_follows_its_inputs_on_another_stream():
    P = Paged([700, 33, 2000], 2, 128, 32, seed=940)
    Q = queries(3, 8, 128, 16)
    want, wlse = attend(P.cache, Q, P.dtable, P.dlens, 0.1)
    n = bg.bi_paged_decode_attention_workspace_bytes(3, 8, 128, P.width * 32)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
    O, lse = torch.empty_like(Q), torch.empty((3, 8), device=DEV)
    Qs, lens = torch.zeros_like(Q), torch.ones_like(P.dlens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        bg.bi_paged_decode_attention(P.cache, Qs, P.dtable, lens, O, 0.1, workspace=ws, lse=lse)
    for _ in range(2):
        ws.fill_(0xFF)
        Qs.copy_(Q)
        lens.copy_(P.dlens)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(O.view(torch.int16), want.view(torch.int16)) and torch.equal(lse, wlse)
        lens.fill_(1)
    with torch.cuda.stream(side):
        bg.bi_paged_decode_attention(P.cache, Q, P.dtable, P.dlens, O, 0.1, workspace=ws, lse=lse)
    side.synchronize()
    assert torch.equal(O.view(torch.int16), want.view(torch.int16))


def test_large_batches():
    # more sequences than a CTA's shared table holds at once, most of them short or empty
    g = np.random.default_rng(17)
    lens = g.integers(0, 70, 2500)
    lens[::100] = 400
    P = Paged(lens, 1, 64, 16, seed=950)
    check(P, 2, 1, 64, seed=18)


@pytest.mark.parametrize("heads,lens", [(8, [1500] * 700), (2, [5000, 1, 0, 300] * 450)])
def test_many_items_per_block(heads, lens):
    # hundreds of chunks for every resident block: their tables are refilled on the way.  All sequences
    # of one length share their pages and queries, so their outputs are equal bit for bit.
    distinct = sorted(set(lens))
    P = Paged(distinct, heads, 64, 64, seed=960)
    row = torch.tensor([distinct.index(n) for n in lens], device=DEV)
    Q = queries(len(distinct), 2 * heads, 64, 19)
    O, lse = attend(P.cache, Q[row].contiguous(), P.dtable[row].contiguous(), P.dlens[row].contiguous(), 0.125)
    one, one_lse = attend(P.cache, Q, P.dtable, P.dlens, 0.125)
    assert torch.equal(O.view(torch.int16), one.view(torch.int16)[row]) and torch.equal(lse, one_lse[row])
    check(P, 2 * heads, heads, 64, seed=19, scale=0.125)


def test_padded_batches_and_empty_tables():
    # a captured batch of 300 slots with a handful in use: the others' rows are zero, or NaN where the
    # length is out of range, and the ones in use do not see them
    P = Paged([700, 3, 260, 1100], 4, 128, 16, seed=970)
    at = [0, 17, 150, 299]
    B = 300
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    table = torch.full((B, P.width), -1, dtype=torch.int32, device=DEV)
    Q = queries(B, 16, 128, 20)
    lens[at], table[at] = P.dlens, P.dtable
    lens[5], lens[200] = -3, 16 * P.width + 1
    O, lse = attend(P.cache, Q, table, lens, 0.1)
    want, wlse = attend(P.cache, Q[at].contiguous(), P.dtable, P.dlens, 0.1)
    assert torch.equal(O[at].view(torch.int16), want.view(torch.int16)) and torch.equal(lse[at], wlse)
    assert torch.isnan(O[[5, 200]].float()).all() and torch.isnan(lse[[5, 200]]).all()
    rest = [b for b in range(B) if b not in at + [5, 200]]
    assert torch.all(O[rest] == 0) and torch.isneginf(lse[rest]).all()
    # no pages at all
    none = torch.empty((B, 0), dtype=torch.int32, device=DEV)
    lens.zero_()
    lens[7] = 1
    O, lse = attend(P.cache, Q, none, lens, 0.1)
    assert torch.isnan(O[7].float()).all() and torch.all(O[:7] == 0) and torch.all(O[8:] == 0)


def test_two_calls_at_once_with_workspaces_of_their_own():
    P = Paged([3000, 40, 900, 2500], 4, 128, 32, seed=980)
    Qs = [queries(4, 16, 128, 21 + i) for i in range(2)]
    want = [attend(P.cache, Q, P.dtable, P.dlens, 0.1)[0] for Q in Qs]
    n = bg.bi_paged_decode_attention_workspace_bytes(4, 16, 128, P.width * 32)
    ws = [torch.empty(n, dtype=torch.uint8, device=DEV) for _ in range(2)]
    outs = [torch.empty_like(Q) for Q in Qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                bg.bi_paged_decode_attention(P.cache, Qs[i], P.dtable, P.dlens, outs[i], 0.1, workspace=ws[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i].view(torch.int16), want[i].view(torch.int16))


def test_back_to_back_steps_in_one_stream_order():
    # write, attend, overwrite and attend again with nothing between them: each attention reads what
    # the write before it left, and the next write does not overtake it
    page, heads, D = 32, 2, 128
    k, v = pool(4, page, heads, D, fill=0), pool(4, page, heads, D, fill=0)
    one = torch.ones((4, heads), device=DEV)
    cache = bg.KvCache(k, v, one, one.clone())
    table = torch.tensor([[2, 0, 3]], dtype=torch.int32, device=DEV)
    slots = torch.tensor([2 * page + i for i in range(page)] + [i for i in range(page)] + [3 * page + i for i in range(9)],
                         dtype=torch.int32, device=DEV)
    n = torch.tensor([2 * page + 9], dtype=torch.int32, device=DEV)
    K = [inputs.bf16_gaussian((2 * page + 9, heads, D), seed=900 + i, device=DEV) for i in range(6)]
    Q = queries(1, 8, D, 22)
    def run(sync):
        outs = []
        for i in range(6):
            bg.bi_kv_append_e4m3(cache, K[i], K[5 - i], slots)
            if sync:
                torch.cuda.synchronize()
            O = torch.empty((1, 8, D), dtype=torch.bfloat16, device=DEV)
            bg.bi_paged_decode_attention(cache, Q, table, n, O, 0.1)
            if sync:
                torch.cuda.synchronize()
            outs.append(O)
        return torch.stack(outs)
    apart = run(True)
    assert len({tuple(o.flatten()[:16].tolist()) for o in apart}) == 6
    for _ in range(5):
        assert torch.equal(run(False).view(torch.int16), apart.view(torch.int16))
