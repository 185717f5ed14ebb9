"""Paged caches for the tests: pools with guard codes around them, tables, and error bounds."""
from __future__ import annotations

import math

import numpy as np
import torch

import invariant_deterministic_gemm_bi_b200 as bg
from invariant_deterministic_gemm_bi_b200 import inputs
from oracle import kv_cache as okv

DEV = "cuda"
NAN_CODE = 0x7F


def pool(pages, page, heads, dim, layout="token", fill=NAN_CODE, device=DEV):
    """uint8 [pages, page, heads, dim]; layout "token": [page][token][head][d], "head": [page][head]
    [token][d], "wide": the token layout inside a wider pool (every stride larger than needed)."""
    if layout == "head":
        return torch.full((pages, heads, page, dim), fill, dtype=torch.uint8, device=device).transpose(1, 2)
    if layout == "wide":
        t = torch.full((pages, page + 2, heads + 1, dim + 16), fill, dtype=torch.uint8, device=device)
        return t[:, :page, :heads, :dim]
    return torch.full((pages, page, heads, dim), fill, dtype=torch.uint8, device=device)


def gaussian_codes(shape, seed, device=DEV):
    return inputs.e4m3_gaussian(shape, seed=seed, device=device).view(torch.uint8)


class Paged:
    """A cache whose sequences' pages are scattered over the pool; every code no sequence owns is NaN
    and every table entry behind a sequence's pages is out of range."""

    def __init__(self, lens, heads, dim, page, seed, layout="token", scales="mixed", spare=2):
        lens = [int(n) for n in lens]
        need = [-(-n // page) for n in lens]
        self.pages, self.page, self.lens = sum(need) + spare, page, lens
        g = np.random.default_rng(seed)
        order = g.permutation(self.pages)
        self.width = max(need + [1]) + 1
        self.table = np.full((len(lens), self.width), 0x7FFFFFF0, np.int32)
        self.table[:, 1::2] = -7
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.k, self.v = pool(self.pages, page, heads, dim, layout), pool(self.pages, page, heads, dim, layout)
        codes = [gaussian_codes((self.pages, page, heads, dim), seed + i) for i in (1, 2)]
        owned = torch.zeros((self.pages, page), dtype=torch.bool)
        for b, n in enumerate(lens):
            for j in range(need[b]):
                owned[self.table[b, j], :min(page, n - j * page)] = True
        owned = owned.to(DEV)[:, :, None, None]
        self.k.copy_(torch.where(owned, codes[0], NAN_CODE))
        self.v.copy_(torch.where(owned, codes[1], NAN_CODE))
        if scales == "one":
            s = [torch.ones((self.pages, heads)), torch.ones((self.pages, heads))]
        elif scales == "pow2":
            s = [inputs.scales_pow2((self.pages, heads), seed + 3 + i, lo=-3, hi=3) for i in range(2)]
        else:   # any positive scale is allowed in the attention
            s = [inputs.scales_log_uniform((self.pages, heads), seed + 3 + i, -2.0, 2.0) for i in range(2)]
        self.k_scale, self.v_scale = s[0].to(DEV), s[1].to(DEV)
        self.cache = bg.KvCache(self.k, self.v, self.k_scale, self.v_scale)
        self.dtable = torch.from_numpy(self.table).to(DEV)
        self.dlens = torch.tensor(lens, dtype=torch.int32, device=DEV)

    def values(self):
        out = []
        for codes, scale in ((self.k, self.k_scale), (self.v, self.v_scale)):
            c = okv.Cache(codes.cpu().numpy(), scale.cpu().numpy())
            out.append(c.dequantised())
        return out


def attend(cache, Q, table, lens, scale, window=0, lse=True, out=None):
    B, Hq, D = Q.shape
    O = torch.full((B, Hq, D), float("nan"), dtype=torch.bfloat16, device=DEV) if out is None else out
    L = torch.full((B, Hq), 7.0, dtype=torch.float32, device=DEV) if lse else None
    n = bg.bi_paged_decode_attention_workspace_bytes(B, Hq, D, table.shape[1] * cache.page_size)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV) if n else None   # NaN wherever unwritten
    bg.bi_paged_decode_attention(cache, Q, table, lens, O, scale, workspace=ws, lse=L, window=window)
    torch.cuda.synchronize()
    return O, L


def assert_attention(O, lse, ref, scale, D, what=""):
    """|O - ref| and |lse - ref| within what the number formats allow.

    Scores: products of a bf16 and an e4m3 value are exact in fp32; D additions, each off by at most
    2^-23 (a cut) of sum |q k|, and four roundings of the scaled score give
    ds = 2^-23 (D + 4) |scale| max_j sum_d |q_d k_jd| + 2^-22 max |s|, the last also standing for the
    exponent's argument in base 2.  A weight exp(s - m) is off by ds, by 2^-22 of the exp2 and, where
    it is held in fp16 for the value product, by 2^-11; the sums over positions are fp32 in chains of
    at most 2^13 additions between roundings, 2^-24 each, which random signs keep far below 2^-14.
    So the output is off by at most (2 ds + 2^-11 + 2^-13) sum_j w_j |v_j| before its own rounding,
    2^-8 of its value; lse by ds + 2^-13 + 2^-23 |lse|.  Weights below the formats' range are lost: fp16
    holds (weight x value scale) scaled to a largest of 2^15 in steps of 2^-24, 2^-39 of the largest, so
    each is off by at most 2^-40 of it on a code of up to 448; and fp32 ends at 2^-126 of the largest.
    """
    ro, rl, spread, mass, floor = ref
    o = O.double().cpu().numpy()
    smax = np.where(np.isfinite(rl), np.abs(rl), 0.0) + 20.0
    ds = 2.0 ** -23 * (D + 4) * abs(scale) * mass + 2.0 ** -22 * smax
    bound = 2.0 ** -8 * np.abs(ro) + (2 * ds[..., None] + 2.0 ** -11 + 2.0 ** -13) * spread * (1 + 2.0 ** -8) + \
        floor[..., None]
    err = np.abs(o - ro)
    assert np.all(err <= bound), (what, float(np.max(err - bound)), np.argwhere(~(err <= bound))[:4])
    if lse is not None:
        l = lse.double().cpu().numpy()
        fin = np.isfinite(rl)
        assert np.array_equal(np.isneginf(l), np.isneginf(rl)), what
        lerr = np.abs(l[fin] - rl[fin])
        lbound = ds[fin] + 2.0 ** -13 + 2.0 ** -23 * np.abs(rl[fin])
        assert np.all(lerr <= lbound), (what, float(np.max(lerr - lbound)))


def queries(B, Hq, D, seed, std=1.0):
    return inputs.bf16_gaussian((B, Hq, D), seed=seed, std=std, device=DEV)


def softmax_scale(D):
    return 1.0 / math.sqrt(D)
