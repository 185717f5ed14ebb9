"""The paged cache's block tables and write on the GPU, bit for bit against the oracle, and a served
run of tables, write and attention together."""
import threading

import numpy as np
import pytest
import torch

import invariant_deterministic_gemm_bi_b200 as bg
from invariant_deterministic_gemm_bi_b200 import inputs
from oracle import kv_cache as okv
from tests.kv_util import DEV, NAN_CODE, assert_attention, attend, pool, softmax_scale

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(np.asarray(v).tolist(), dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------------------------------------
# block tables
# ---------------------------------------------------------------------------------------------

def run_tables(ctx, new, page, stack, count, table, max_tokens, positions=True):
    B = len(ctx)
    s = {"stack": ints(stack), "table": ints(table), "lens": ints([7] * B), "offsets": ints([7] * (B + 1)),
         "slots": ints([7] * max_tokens), "positions": ints([7] * max_tokens), "left": ints([7]), "status": ints([7])}
    bg.bi_kv_block_tables(ints(ctx), ints(new), page, s["stack"], ints([count]), s["table"], s["lens"], s["offsets"],
                          s["slots"], s["left"], s["status"], positions=s["positions"] if positions else None)
    torch.cuda.synchronize()
    return s


def assert_tables(s, want):
    for k in ("table", "stack", "lens", "offsets", "slots", "positions"):
        assert np.array_equal(s[k].cpu().numpy(), want[k]), k
    assert s["left"].item() == want["left"] and s["status"].item() == want["status"]


def scenario(B, page, top_ctx, top_new, seed, ended=0.2, spare=3, pad=5):
    g = np.random.default_rng(seed)
    ctx = g.integers(0, top_ctx + 1, B)
    new = np.where(g.random(B) < 0.5, 1, g.integers(0, top_new + 1, B))
    new[g.random(B) < ended] = -1
    have = -(-ctx // page)
    need = np.where(new < 0, 0, -(-(ctx + new.clip(0)) // page) - have)
    width = int((have + need).max()) if B else 1
    pages = g.permutation(int(have.sum() + need.sum()) + spare)
    table = np.full((B, max(width, 1)), -3)
    table[np.arange(table.shape[1]) < have[:, None]] = pages[:have.sum()]
    free = pages[have.sum():]
    stack = np.full(free.size + int(have[new < 0].sum()), -5)
    stack[:free.size] = free
    return ctx, new, page, stack, free.size, table, int(new.clip(0).sum()) + pad


@pytest.mark.parametrize("B,page,top_ctx,top_new", [
    (1, 16, 0, 1), (1, 256, 1000, 700), (3, 32, 40, 0), (31, 16, 50, 40), (64, 16, 4096, 1), (257, 128, 3000, 300),
    (1000, 64, 2000, 1), (1025, 16, 100, 60), (5000, 32, 64, 20), (8192, 16, 40, 3)])
def test_tables_match_the_oracle(B, page, top_ctx, top_new):
    a = scenario(B, page, top_ctx, top_new, seed=B + page)
    s = run_tables(*a)
    assert_tables(s, okv.block_tables(*a))


def test_tables_of_long_prompts():
    a = scenario(7, 16, 0, 60000, seed=5, ended=0.0)
    assert_tables(run_tables(*a), okv.block_tables(*a))


def test_tables_without_positions_requests_or_tokens():
    a = scenario(9, 16, 100, 5, seed=6)
    s = run_tables(*a, positions=False)
    assert torch.all(s["positions"] == 7)
    assert np.array_equal(s["slots"].cpu().numpy(), okv.block_tables(*a)["slots"])
    empty = ([], [], 16, [1, 2, 3], 2, np.zeros((0, 4), int), 3)
    s = {k: ints(v) for k, v in {"stack": [1, 2, 3], "offsets": [7], "slots": [7] * 3, "left": [7], "status": [7]}.items()}
    z = torch.zeros((0, 4), dtype=torch.int32, device=DEV)
    bg.bi_kv_block_tables(ints([]), ints([]), 16, s["stack"], ints([2]), z, ints([]), s["offsets"], s["slots"], s["left"],
                          s["status"])
    want = okv.block_tables(*empty)
    assert s["slots"].tolist() == [-1] * 3 and s["offsets"].tolist() == [0] and s["left"].item() == want["left"] == 2
    # nobody has new tokens: no slot rows at all
    a = ([5, 40], [0, -1], 16, [9, 9, 9, 9], 1, np.array([[0, -1, -1], [1, 2, 3]]), 0)
    assert_tables(run_tables(*a), okv.block_tables(*a))


BASE = dict(ctx=[20, 9, 0, 33], new=[13, -1, 17, 0], page=16, stack=[2, 4, 6, 8, -1], count=4,
            table=np.array([[7, 3, -9, -9], [5, -9, -9, -9], [-9] * 4, [1, 10, 11, -9]]), max_tokens=32)


@pytest.mark.parametrize("change", [
    {"ctx": [20, -9, 0, 33]}, {"new": [13, -2, 17, 0]}, {"count": 6}, {"count": -1}, {"new": [45, -1, 17, 0]},
    {"max_tokens": 29}, {"count": 1}, {"count": 5}, {"ctx": [20, 65, 0, 33]}, {"new": [2 ** 31 - 1] * 4},
    {"new": [2 ** 31 - 1, -1, 1, 1], "ctx": [2 ** 31 - 1, 0, 0, 0]}])
def test_what_does_not_fit_changes_nothing(change):
    a = list((BASE | change).values())
    want = okv.block_tables(*a)
    assert want["status"] != 0
    assert_tables(run_tables(*a), want)
    good = list(BASE.values())
    assert okv.block_tables(*good)["status"] == 0


def test_bad_page_numbers_on_the_stack_give_no_slot():
    a = ([0, 0, 0], [1, 1, 1], 256, [3, -4, 2 ** 31 - 1], 3, np.full((3, 1), -1), 3)
    s = run_tables(*a)
    assert s["slots"].tolist() == [-1, -1, 3 * 256] and s["status"].item() == 0


def test_host_threads_with_different_numbers_of_requests():
    """Each call needs shared memory for its own requests; one thread's amount must not become the other's."""
    failures = []

    def work(B):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                ctx, new, lens, offsets = ints([5] * B), ints([0] * B), ints([7] * B), ints([7] * (B + 1))
                table, stack, one, slots = ints([[3]] * B), ints([4]), ints([1]), ints([7])
                left, status = ints([7]), ints([7])
                for _ in range(2000):
                    bg.bi_kv_block_tables(ctx, new, 16, stack, one, table, lens, offsets, slots, left, status)
                torch.cuda.current_stream().synchronize()
            assert torch.all(lens == 5) and left.item() == 1 and status.item() == 0
        except Exception as e:   # reported by the test's own thread
            failures.append((B, e))

    threads = [threading.Thread(target=work, args=(B,)) for B in (3500, 5000, 8192)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures


def test_lengths_and_count_in_place_under_a_replayed_graph():
    # a decode step captured once: the lengths and the stack live in the buffers it updates.  Near the
    # end the nine pages it asks for are more than the eight on the stack: such a step changes nothing
    B, page = 5, 16
    ctx0 = [15, 16, 31, 0, 3]
    table0 = np.full((B, 4), -1)
    table0[0, 0], table0[1, 0], table0[2, :2], table0[4, 0] = 4, 9, [1, 7], 2
    stack0 = [11, 12, 13, 14, 15, 16, 17, 18]
    ctx, table, stack, count = ints(ctx0), ints(table0), ints(stack0), ints([8])
    offsets, slots, status, new = ints([0] * (B + 1)), ints([0] * B), ints([9]), ints([1] * B)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bg.bi_kv_block_tables(ctx, new, page, stack, count, table, ctx, offsets, slots, count, status)
    want = {"lens": np.array(ctx0), "table": table0, "stack": np.array(stack0), "left": 8}
    for step in range(20):
        graph.replay()
        want = okv.block_tables(want["lens"], [1] * B, page, want["stack"], want["left"], want["table"], B)
        assert slots.tolist() == want["slots"].tolist() and ctx.tolist() == want["lens"].tolist()
        assert np.array_equal(table.cpu().numpy(), want["table"]) and count.item() == want["left"]
        assert status.item() == want["status"]
    assert want["status"] == okv.UNSUPPORTED


# ---------------------------------------------------------------------------------------------
# the write
# ---------------------------------------------------------------------------------------------

def fresh(pages, page, heads, dim, layout="token"):
    k, v = pool(pages, page, heads, dim, layout), pool(pages, page, heads, dim, layout)
    ks, vs = torch.full((pages, heads), 3.0, device=DEV), torch.full((pages, heads), 3.0, device=DEV)
    return bg.KvCache(k, v, ks, vs)


def tokens(T, heads, dim, seed, spread=3.0):
    """bf16 rows whose magnitudes differ by 2^(spread N(0, 1)) from token to token and head to head."""
    x = inputs.bf16_gaussian((T, heads, dim), seed=seed, device=DEV).float()
    g = inputs.generator(seed + 1, DEV)
    return (x * torch.exp2(spread * torch.randn((T, heads, 1), generator=g, device=DEV))).to(torch.bfloat16)


def assert_pool(codes, scales, want):
    got = okv.Cache(codes.cpu().numpy(), scales.cpu().numpy())
    assert np.array_equal(got.scale, want.scale), np.argwhere(got.scale != want.scale)[:4]
    assert np.array_equal(got.value, want.value, equal_nan=True), np.argwhere(~((got.value == want.value) | np.isnan(want.value)))[:4]


def write_and_compare(cache, K, V, slots, pieces=None):
    want = [okv.Cache(c.cpu().numpy(), s.cpu().numpy()) for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]
    want[0].append(inputs.to_numpy_bits(K), slots)
    want[1].append(inputs.to_numpy_bits(V), slots)
    at = 0
    for n in pieces or [len(slots)]:
        bg.bi_kv_append_e4m3(cache, K[at:at + n], V[at:at + n], ints(slots[at:at + n]))
        at += n
    torch.cuda.synchronize()
    assert_pool(cache.k, cache.k_scale, want[0])
    assert_pool(cache.v, cache.v_scale, want[1])


def prompt_slots(pages, start, n, page):
    pos = np.arange(start, start + n)
    return (np.asarray(pages)[pos // page] * page + pos % page).tolist()


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("heads,dim,layout", [(1, 128, "token"), (3, 64, "head"), (2, 128, "wide")])
def test_prompts_and_pieces_match_the_oracle(page, heads, dim, layout):
    cache = fresh(12, page, heads, dim, layout)
    slots = prompt_slots([7, 2, 5], 0, 2 * page + 9, page) + [-1, -1] + prompt_slots([0], 0, 1, page) + \
        prompt_slots([11, 4], 0, page + 1, page)
    write_and_compare(cache, tokens(len(slots), heads, dim, 31 + page), tokens(len(slots), heads, dim, 32 + page), slots)
    # more tokens behind them: a piece that ends inside a page, one that crosses into a new one, single ones
    slots = prompt_slots([7, 2, 5], 2 * page + 9, 5, page) + prompt_slots([0], 1, page - 1, page) + \
        prompt_slots([11, 4, 8], page + 1, page, page) + [12 * page, -3, 2 ** 31 - 1]
    write_and_compare(cache, tokens(len(slots), heads, dim, 33 + page), tokens(len(slots), heads, dim, 34 + page, 6.0), slots)


def test_the_calls_that_wrote_a_page_do_not_matter():
    page, heads, dim, n = 32, 2, 128, 77
    K, V = tokens(n, heads, dim, 41, 5.0), tokens(n, heads, dim, 43, 5.0)
    slots = prompt_slots([3, 0, 2], 0, n, page)
    caches = []
    for pieces in ([n], [1] * n, [5, 40, 1, 1, 30], [33, 44]):
        c = fresh(4, page, heads, dim)
        write_and_compare(c, K, V, slots, pieces)
        caches.append(c)
    for c in caches[1:]:
        assert torch.equal(c.k, caches[0].k) and torch.equal(c.v, caches[0].v)
        assert torch.equal(c.k_scale, caches[0].k_scale) and torch.equal(c.v_scale, caches[0].v_scale)
    # writing a page's last tokens again changes nothing
    before = caches[0].k.clone()
    bg.bi_kv_append_e4m3(caches[0], K[70:], V[70:], ints(slots[70:]))
    assert torch.equal(caches[0].k, before)


def test_every_code_decision():
    # all bf16 magnitudes within the page's range, both signs: ties, subnormals, the cut, saturation
    page, heads, dim = 256, 1, 128
    bits = torch.arange(page * dim, dtype=torch.int32).to(torch.int16).view(page, heads, dim)
    K = bits.view(torch.bfloat16).to(DEV)          # 0x0000 .. 0x7fff: every positive bf16, inf and NaN
    V = (-K.float()).to(torch.bfloat16)
    slots = list(range(page))
    write_and_compare(fresh(1, page, heads, dim), K, V, slots)
    # magnitudes around one scale, where every decision of R lies
    x = torch.from_numpy(np.float32(2.0) ** np.linspace(-20, 8.8, page * dim)).to(torch.bfloat16).view(page, heads, dim)
    x = x.to(DEV)
    x[0] = 448.0
    write_and_compare(fresh(1, page, heads, dim), x, -x, slots)


@pytest.mark.parametrize("value", [0.0, -0.0, 1e-38, 1e-41, float("inf"), float("nan"), 3.38e38, 448.0 * 2.0 ** 64])
def test_extreme_tokens(value):
    cache = fresh(2, 16, 2, 64)
    K, V = tokens(5, 2, 64, 51), tokens(5, 2, 64, 52)
    K[0], V[2] = value, value                       # a first token, and one behind others
    K[3, 1, 5] = value
    write_and_compare(cache, K, V, [16, 17, 18, 19, 20])


def test_rows_of_a_projection_and_untouched_pages():
    # K and V are slices of one wider row, straight from the GEMM
    heads, dim, T, hidden = 2, 128, 37, 256
    plan = bg.bi_gemm_plan(8 * dim, hidden)
    X = inputs.bf16_gaussian((T, hidden), seed=61, device=DEV)
    W = inputs.bf16_gaussian((8 * dim, hidden), seed=62, std=hidden ** -0.5, device=DEV)
    C = torch.empty((T, 8 * dim), dtype=torch.bfloat16, device=DEV)
    bg.bi_gemm_run(plan, X, W, C)
    K, V = C[:, 4 * dim:6 * dim].view(T, heads, dim), C[:, 6 * dim:].view(T, heads, dim)
    cache = fresh(6, 16, heads, dim)
    write_and_compare(cache, K, V, prompt_slots([4, 1, 2], 3, T, 16))
    for p in (0, 3, 5):
        assert torch.all(cache.k[p] == NAN_CODE) and torch.all(cache.v[p] == NAN_CODE)
        assert torch.all(cache.k_scale[p] == 3.0)
    assert torch.all(cache.k[4, :3] == NAN_CODE)    # places before the run: NaN stays NaN


def test_many_single_tokens_and_no_tokens():
    page, heads, dim, B = 64, 8, 128, 300
    cache = fresh(B, page, heads, dim)
    off = np.random.default_rng(71).integers(0, page, B)
    slots = (np.random.default_rng(72).permutation(B) * page + off).tolist()
    cache.k.copy_(inputs.e4m3_gaussian(cache.k.shape, 73, DEV).view(torch.uint8))
    cache.v.copy_(inputs.e4m3_gaussian(cache.v.shape, 74, DEV).view(torch.uint8))
    cache.k_scale.copy_(inputs.scales_pow2((B, heads), 75, device=DEV))
    cache.v_scale.copy_(inputs.scales_pow2((B, heads), 76, device=DEV))
    write_and_compare(cache, tokens(B, heads, dim, 77), tokens(B, heads, dim, 78), slots)
    empty = torch.empty((0, heads, dim), dtype=torch.bfloat16, device=DEV)
    bg.bi_kv_append_e4m3(cache, empty, empty, ints([]))


@pytest.mark.parametrize("page,heads,dim,B", [(128, 2, 64, 1200), (16, 2, 128, 2500), (256, 1, 64, 900)])
def test_large_steps_of_single_tokens_and_pieces(page, heads, dim, B):
    # so many rows that a block holds 32 of them: single tokens beside runs of a few, runs that cross
    # the middle of a block and its end, and skipped rows, each request in a page of its own
    g = np.random.default_rng(page + B)
    cache = fresh(B, page, heads, dim)
    cache.k.copy_(inputs.e4m3_gaussian(cache.k.shape, 91, DEV).view(torch.uint8))
    cache.v.copy_(inputs.e4m3_gaussian(cache.v.shape, 92, DEV).view(torch.uint8))
    cache.k_scale.copy_(inputs.scales_pow2((B, heads), 93, lo=-6, hi=2, device=DEV))
    cache.v_scale.copy_(inputs.scales_pow2((B, heads), 94, lo=-6, hi=2, device=DEV))
    slots = []
    for p in g.permutation(B):
        n = min(int(g.choice([1, 1, 1, 1, 2, 3, 5, 17, 40])), page)
        off = int(g.integers(0, page - n + 1)) if g.random() < 0.8 else 0
        slots += [int(p) * page + off + i for i in range(n)] + [-1] * int(g.integers(0, 2))
    write_and_compare(cache, tokens(len(slots), heads, dim, 95, 2.0), tokens(len(slots), heads, dim, 97, 2.0), slots)


def test_slots_beyond_32_bits_of_codes():
    page, heads, dim = 256, 8, 128
    pages = (9 << 29) // (page * heads * dim)
    cache = fresh(pages, page, heads, dim)
    slots = prompt_slots([pages - 1, 0, pages - 2], 200, 100, page)
    K, V = tokens(100, heads, dim, 81), tokens(100, heads, dim, 82)
    small = fresh(3, page, heads, dim)
    bg.bi_kv_append_e4m3(cache, K, V, ints(slots))
    bg.bi_kv_append_e4m3(small, K, V, ints(prompt_slots([0, 1, 2], 200, 100, page)))
    at = [pages - 1, 0, pages - 2]
    assert torch.equal(cache.k[at], small.k) and torch.equal(cache.v[at], small.v)
    assert torch.equal(cache.k_scale[at], small.k_scale) and torch.equal(cache.v_scale[at], small.v_scale)
    assert torch.all(cache.k[pages // 2] == NAN_CODE)


# ---------------------------------------------------------------------------------------------
# all of it, as a server runs it
# ---------------------------------------------------------------------------------------------

@pytest.mark.parametrize("page,dim,Hq,heads", [(16, 64, 6, 2), (32, 128, 8, 1)])
def test_a_served_run(page, dim, Hq, heads):
    """Twelve steps of six request slots: prompts in pieces, decodes, ends and new requests in the
    freed pages; every step's cache and attention against the oracle, and every request's last
    output bit for bit against the same request served alone in one prompt."""
    B, width, pages, steps = 6, 8, 24, 12
    g = np.random.default_rng(page)
    cache = fresh(pages, page, heads, dim)
    table = ints(np.full((B, width), -1))
    stack, count, status = ints(g.permutation(pages)), ints([pages]), ints([0])
    lens, offsets = ints([0] * B), ints([0] * (B + 1))
    T = 160
    slots, positions = ints([0] * T), ints([0] * T)
    plan_new = [[40, 0, 7, 1, 0, 0], [1, 3, 1, 1, 0, 60], [1, 30, 1, 1, 0, 30], [1, 1, -1, 1, 9, 1], [1, 1, 0, 1, 1, 1],
                [1, 1, 50, -1, 1, 1], [1, -1, 1, 0, 1, 1], [1, 17, 1, 2, 1, -1], [-1, 1, 1, 1, 1, 0], [33, 1, 1, 1, 1, 5],
                [1, 1, 1, 1, 1, 1], [1, 1, 1, 1, 1, 1]]
    oracle_k = okv.Cache(cache.k.cpu().numpy(), cache.k_scale.cpu().numpy())
    oracle_v = okv.Cache(cache.v.cpu().numpy(), cache.v_scale.cpu().numpy())
    state = {"lens": np.zeros(B, int), "table": table.cpu().numpy(), "stack": stack.cpu().numpy(), "left": pages}
    history = [([], []) for _ in range(B)]
    scale = softmax_scale(dim)
    for step in range(steps):
        new = plan_new[step]
        K, V = tokens(T, heads, dim, 1000 + step, 1.5), tokens(T, heads, dim, 2000 + step, 1.5)
        Q = inputs.bf16_gaussian((B, Hq, dim), seed=3000 + step, device=DEV)
        bg.bi_kv_block_tables(lens, ints(new), page, stack, count, table, lens, offsets, slots, count, status,
                              positions=positions)
        bg.bi_kv_append_e4m3(cache, K, V, slots)
        O, lse = attend(cache, Q, table, lens, scale)
        state = okv.block_tables(state["lens"], new, page, state["stack"], state["left"], state["table"], T)
        assert status.item() == state["status"] == 0
        assert np.array_equal(table.cpu().numpy(), state["table"]) and count.item() == state["left"]
        assert np.array_equal(slots.cpu().numpy(), state["slots"])
        oracle_k.append(inputs.to_numpy_bits(K), state["slots"])
        oracle_v.append(inputs.to_numpy_bits(V), state["slots"])
        assert_pool(cache.k, cache.k_scale, oracle_k)
        assert_pool(cache.v, cache.v_scale, oracle_v)
        ref = okv.paged_attention(inputs.to_numpy_bits(Q), oracle_k.dequantised(), oracle_v.dequantised(), state["table"],
                                  state["lens"], scale, v_scale=oracle_v.scale)
        assert_attention(O, lse, ref, scale, dim, f"step {step}")
        for b in range(B):
            if new[b] < 0:
                history[b] = ([], [])
            else:
                rows = slice(state["offsets"][b], state["offsets"][b + 1])
                history[b][0].append(K[rows])
                history[b][1].append(V[rows])
    for b in range(B):
        K, V = torch.cat(history[b][0]), torch.cat(history[b][1])
        n = K.shape[0]
        assert n == state["lens"][b] > 0
        alone = fresh(width, page, heads, dim)
        row = list(range(width))
        bg.bi_kv_append_e4m3(alone, K, V, ints(prompt_slots(row, 0, n, page)))
        Oa, la = attend(alone, Q[b:b + 1], ints([row]), ints([n]), scale)
        assert torch.equal(Oa.view(torch.int16)[0], O.view(torch.int16)[b]) and torch.equal(la[0], lse[b])
