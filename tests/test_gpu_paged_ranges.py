"""Decode attention over the paged 8-bit cache at the ends of the ranges that its header allows:
scores of any finite size, value scales far apart, factors beyond fp32 on scores inside it."""
import numpy as np
import pytest
import torch

import invariant_deterministic_gemm_bi_b200 as bg
from invariant_deterministic_gemm_bi_b200 import inputs
from oracle import kv_cache as okv
from tests.kv_util import DEV, assert_attention, attend, gaussian_codes, pool, queries

pytestmark = pytest.mark.gpu
ONE = 0x38   # e4m3 code of 1.0


def sequence(n, heads, dim, page, seed, k_scale=1.0, v_scale=1.0):
    """One sequence of n positions in the pages 0, 1, ...: zero keys, gaussian values."""
    pages = -(-n // page)
    k = pool(pages, page, heads, dim, fill=0)
    v = gaussian_codes((pages, page, heads, dim), seed)
    ks = torch.full((pages, heads), k_scale, device=DEV)
    vs = torch.full((pages, heads), v_scale, device=DEV)
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None].contiguous()
    return bg.KvCache(k, v, ks, vs), table, torch.tensor([n], dtype=torch.int32, device=DEV)


def oracle(cache, Q, table, lens, scale):
    K, V = (okv.Cache(c.cpu().numpy(), s.cpu().numpy()).dequantised()
            for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
    return okv.paged_attention(inputs.to_numpy_bits(Q), K, V, table.cpu().numpy(), lens.tolist(), scale,
                               v_scale=cache.v_scale.cpu().numpy())


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("top", [2.0 ** 23, 1.3 * 2.0 ** 24, 1.9 * 2.0 ** 24, 2.0 ** 25 + 8, 1.1 * 2.0 ** 27, 2.0 ** 30, 2.0 ** 100])
def test_equal_scores_of_any_size(top, sign):
    """Equal keys: the weights are 1 / n whatever the score, so the output is the mean value, off by 2^-8
    of its own rounding and 2^-11 of the mean magnitude (fp16 weights; fp32 sums of at most 600 terms are
    far below that), and the log-sum-exp is the score + log n, off by four fp32 roundings."""
    for n in (1, 40, 600):
        cache, table, lens = sequence(n, 2, 128, 32, seed=n)
        cache.k.fill_(ONE)
        Q = torch.ones((1, 8, 128), dtype=torch.bfloat16, device=DEV)
        scale = sign * top / (128 * 1.4426950408889634)
        O, lse = attend(cache, Q, table, lens, scale)
        v = cache.v.view(torch.float8_e4m3fn).double().reshape(-1, 2, 128)[:n]
        want, spread = v.mean(0), v.abs().mean(0)
        got = O[0].double().view(2, 4, 128)
        bound = 2.0 ** -8 * want.abs() + 2.0 ** -11 * (1 + 2.0 ** -8) * spread
        assert torch.all((got - want[:, None]).abs() <= bound[:, None]), n
        s = 128 * float(np.float32(scale))
        assert torch.all((lse.double() - (s + np.log(n))).abs() <= 2.0 ** -22 * (abs(s) + np.log(n)) + 2.0 ** -20), n


@pytest.mark.parametrize("dim", [64, 128])
def test_large_scores_that_differ(dim):
    """Scores 2^27 to 2^29 and thousands apart: the largest alone counts, its value comes out exactly."""
    n = 700
    cache, table, lens = sequence(n, 1, dim, 64, seed=5)
    codes = torch.randint(1, 0x60, (n,), generator=inputs.generator(6, DEV), device=DEV).to(torch.uint8)
    codes[codes == 0x5F] = 0x5E
    at = torch.tensor([0, 31, 300, 699], device=DEV)
    for best in at.tolist():
        c = codes.clone()
        c[best] = 0x5F
        cache.k.view(-1, 1, dim)[:n, 0, 0] = c
        Q = torch.zeros((1, 4, dim), dtype=torch.bfloat16, device=DEV)
        Q[..., 0] = 2.0 ** 20
        O, lse = attend(cache, Q, table, lens, 8.0)
        v = cache.v.view(torch.float8_e4m3fn).view(-1, dim)[best].to(torch.bfloat16)
        assert torch.equal(O[0], v.expand(4, -1)), best
        s = 2.0 ** 23 * float(torch.tensor([0x5F], dtype=torch.uint8).view(torch.float8_e4m3fn).double())
        assert torch.all((lse.double() - s).abs() <= 2.0 ** -22 * s)


def log2_keys(cache, rows, x):
    """Keys whose score is x in base 2 for a query of ones in dimension 0 and scale 2 ln 2: x / 2 in dimension 0."""
    code = torch.tensor([x / 2], dtype=torch.float32).to(torch.float8_e4m3fn).view(torch.uint8)
    assert float(code.view(torch.float8_e4m3fn).float()) == x / 2
    cache.k.view(-1, cache.num_heads, cache.head_dim)[rows, :, 0] = code.to(DEV)


# (positions, page, head_dim, pages in the large scale, base-2 score of the others below theirs)
FAR = [(17, 16, 64, [1], -14), (17, 16, 128, [1], -14), (256, 32, 128, [0], 0), (256, 32, 64, [5], -8),
       (256, 32, 128, [7], -16), (2000, 64, 64, [0], 0), (2000, 64, 128, [31], -4), (9000, 256, 64, [17], -8),
       (131072 + 256, 256, 64, [0], -14), (131072 + 256, 256, 64, [512], -14), (20000, 16, 128, [3, 700], -20)]


@pytest.mark.parametrize("n,page,dim,large,below", FAR)
@pytest.mark.parametrize("far", [64, 63.5])
def test_value_scales_at_both_ends_of_their_range(n, page, dim, large, below, far):
    # positions of a small value scale add nothing to the output, but all of them to the softmax sum
    cache, table, lens = sequence(n, 1, dim, page, seed=11, v_scale=2.0 ** -far)
    log2_keys(cache, slice(None), below)
    for p in large:
        cache.v_scale[p] = 2.0 ** far
        cache.k[p] = 0
    Q = torch.zeros((1, 4, dim), dtype=torch.bfloat16, device=DEV)
    Q[..., 0] = 1
    scale = 2 * np.log(2.0)
    O, lse = attend(cache, Q, table, lens, scale)
    assert_attention(O, lse, oracle(cache, Q, table, lens, scale), scale, dim)


@pytest.mark.parametrize("seed", range(4))
def test_value_scales_over_all_of_their_range(seed):
    g = inputs.generator(100 + seed, DEV)
    for n, page, dim, heads in ((77, 16, 64, 2), (700, 16, 128, 1), (5000, 32, 64, 1), (30000, 64, 128, 1)):
        cache, table, lens = sequence(n, heads, dim, page, seed=12 + seed)
        cache.k.copy_(gaussian_codes(cache.k.shape, 13 + seed))
        cache.v_scale.copy_(torch.exp2(torch.randint(-64, 65, cache.v_scale.shape, generator=g, device=DEV).float()))
        Q = queries(1, 4 * heads, dim, 14 + seed, std=3.0)
        O, lse = attend(cache, Q, table, lens, 0.3)
        assert_attention(O, lse, oracle(cache, Q, table, lens, 0.3), 0.3, dim)


@pytest.mark.parametrize("scale,std", [(3e38, 1.0), (-3e38, 30.0), (2.4e38, 1e-3), (1e30, 1e30), (1e38, 1e38)])
def test_zero_keys_have_score_zero_whatever_the_factors(scale, std):
    cache, table, lens = sequence(300, 2, 128, 32, seed=21, k_scale=2.0 ** -64)
    cache.k_scale[3:5] = 2.0 ** 64
    Q = queries(1, 8, 128, 22, std=std)
    O, lse = attend(cache, Q, table, lens, scale)
    assert_attention(O, lse, oracle(cache, Q, table, lens, scale), 0.0, 128)


@pytest.mark.parametrize("scale,q,k_scale", [(3e38, 2.0 ** 20, 2.0 ** -64), (2.4e38, 1.0, 2.0 ** -40), (1e30, 2.0 ** 60, 2.0 ** -64),
                                             (1e25, 2.0 ** 80, 2.0 ** -60), (-3e38, 2.0 ** 30, 2.0 ** -64)])
def test_scores_inside_fp32_of_factors_beyond_it(scale, q, k_scale):
    """scale * log2 e * |q| is beyond fp32 or near its end, the scores are not: distinct keys, the largest
    score alone counts."""
    n = 200
    cache, table, lens = sequence(n, 1, 64, 16, seed=23, k_scale=k_scale)
    rows = cache.k.view(-1, 1, 64)
    rows[:n, 0, 0] = torch.randint(8, 40, (n,), generator=inputs.generator(24, DEV), device=DEV).to(torch.uint8)
    for best in (0, 17, 133, 199):
        codes = rows[:n, 0, 0].clone()
        rows[best, 0, 0] = 48 if scale > 0 else 4
        Q = torch.zeros((1, 2, 64), dtype=torch.bfloat16, device=DEV)
        Q[..., 0], Q[0, 1, 5] = q, 1e-3
        s = float(np.float32(scale)) * q * k_scale * float(rows[best:best + 1, 0, 0].view(torch.float8_e4m3fn).double())
        assert abs(s) * 1.5 < 3e38
        O, lse = attend(cache, Q, table, lens, scale)
        v = cache.v.view(torch.float8_e4m3fn).view(-1, 64)[best].to(torch.bfloat16)
        assert torch.equal(O[0], v.expand(2, -1)), best
        assert torch.all((lse.double() - s).abs() <= 2.0 ** -21 * abs(s))
        rows[:n, 0, 0] = codes


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("down,scale", [(28, 2.0 ** 28), (20, 2.0 ** 20), (34, 2.0 ** 30)])
def test_small_entries_beside_a_large_one_that_meets_zero_keys(dim, down, scale):
    """Entries down to 2^-28 of the head's largest are exact; below, a score is off by up to scale * 2^-39 of the
    largest times sum |k|, which moves a weight by as much."""
    cache, table, lens = sequence(400, 1, dim, 32, seed=25)
    cache.k.copy_(gaussian_codes(cache.k.shape, 26))
    cache.k[..., 0] = 0
    Q = (queries(1, 4, dim, 27).float().clamp(-1.9, 1.9) * 2.0 ** -down).to(torch.bfloat16)
    if down == 28:   # magnitudes in [1, 2), so that every entry is at or above 2^-28
        Q = (Q.float() + torch.sign(Q.float()) * 2.0 ** -down).clamp(-1.99 * 2.0 ** -down, 1.99 * 2.0 ** -down).to(torch.bfloat16)
    Q[..., 0] = 1
    O, lse = attend(cache, Q, table, lens, scale)
    ref = list(oracle(cache, Q, table, lens, scale))
    if down > 28:
        k = okv.Cache(cache.k.cpu().numpy(), cache.k_scale.cpu().numpy()).dequantised()
        # ds = 2^-23 (D + 4) |scale| mass in the bound: mass grows by what the entries may be off
        ref[3] = ref[3] + np.abs(k).sum(-1).max() * 2.0 ** -39 * 2.0 ** 23 / (dim + 4)
    assert_attention(O, lse, ref, scale, dim)
