"""Block tables of batches whose request slots are mostly idle (no new tokens), a server's ordinary state."""
import numpy as np
import pytest
import torch

import invariant_deterministic_gemm_bi_b200 as bg
from oracle import kv_cache as okv
from tests.test_gpu_kv_cache import assert_tables, ints, run_tables

pytestmark = pytest.mark.gpu


def batch(B, used, most_new, seed, ended=0):
    """Arguments of run_tables: `used` of B requests get 1 to most_new tokens, `ended` others end."""
    g = np.random.default_rng(seed)
    ctx = g.integers(0, 50, B)
    new = np.zeros(B, int)
    pick = g.permutation(B)
    new[pick[:used]] = g.integers(1, most_new + 1, used)
    new[pick[used:used + ended]] = -1
    have = -(-ctx // 16)
    need = np.where(new < 0, 0, -(-(ctx + new.clip(0)) // 16) - have)
    pages = g.permutation(int(have.sum() + need.sum()) + 3)
    table = np.full((B, int((have + need).max()) + 1), -3)
    table[np.arange(table.shape[1]) < have[:, None]] = pages[:have.sum()]
    free = pages[have.sum():]
    stack = np.concatenate([free, np.full(int(have[new < 0].sum()), -5)])
    return ctx, new, 16, stack, free.size, table, int(new.clip(0).sum()) + 5


@pytest.mark.parametrize("B,used,most_new,ended", [
    (8192, 1, 1, 0), (8192, 2, 1, 5), (8192, 16, 1, 0), (8192, 16, 9, 100), (8192, 700, 3, 10), (8192, 4000, 1, 0),
    (1000, 3, 40, 0), (300, 150, 2, 30), (40, 20, 5, 3), (5, 1, 1, 1)])
def test_idle_requests_between_tokens(B, used, most_new, ended):
    a = batch(B, used, most_new, seed=B + used, ended=ended)
    assert_tables(run_tables(*a), okv.block_tables(*a))


def test_idle_requests_cost_no_walk():
    """The tokens of one thread may belong to requests far apart; the requests between them are searched
    over, not walked over (16 of 8192 slots took six times as long as one)."""
    times = []
    for used in (1, 16):
        ctx, new, page, stack, count, table, T = batch(8192, used, 1, seed=used)
        s = [ints(x) for x in (ctx, new, stack, [count], table, [0] * 8192, [0] * 8193, [0] * T, [0], [0])]

        def call():
            bg.bi_kv_block_tables(s[0], s[1], page, s[2], s[3], s[4], s[5], s[6], s[7], s[8], s[9])
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(20):
                call()
        best = float("inf")
        for _ in range(30):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            graph.replay()
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        times.append(best)
    assert times[1] < 3 * times[0], times
