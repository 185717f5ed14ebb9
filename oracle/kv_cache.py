"""CPU oracle for the paged 8-bit key/value cache -- TEST INFRASTRUCTURE ONLY.

The definitions of ``include/bi_kv_cache.h`` and ``include/bi_paged_attention.h`` written out in
plain Python integers and numpy fp64: block tables request by request, the write token by token
(every token rounds the codes that are there to the new scale again, so that the order of writing
really happens), attention sequence by sequence.

Pins: ``tests/test_oracle_kv_cache.py``.
"""
from __future__ import annotations

import numpy as np

from .oracle import bf16_to_f64, e4m3_to_f64

E_MIN, E_MAX = -64, 64
OK, INVALID, UNSUPPORTED = 0, 1, 3


def block_tables(ctx, new, page, stack, count, table, max_tokens):
    """The outputs of bi_kv_block_tables as a dict; ``stack`` and ``table`` (numpy) are not changed."""
    ctx, new = [int(x) for x in ctx], [int(x) for x in new]
    stack, table = np.array(stack), np.array(table)
    B, width = table.shape
    pages = lambda n: -(-n // page)
    status = OK
    if any(c < 0 for c in ctx) or any(n < -1 for n in new) or count < 0 or count > stack.size:
        status = INVALID
    else:
        back = sum(pages(c) for c, n in zip(ctx, new) if n < 0)
        need = sum(pages(c + n) - pages(c) for c, n in zip(ctx, new) if n >= 0)
        if (any(pages(c + max(n, 0)) > width for c, n in zip(ctx, new)) or sum(max(n, 0) for n in new) > max_tokens
                or count + back > stack.size or need > count + back):
            status = UNSUPPORTED
    slots, positions = np.full(max_tokens, -1, np.int64), np.full(max_tokens, -1, np.int64)
    if status:
        return {"table": table, "stack": stack, "lens": np.array(ctx), "offsets": np.zeros(B + 1, int),
                "slots": slots, "positions": positions, "left": count, "status": status}
    top = count
    for b in range(B):
        if new[b] < 0:
            for p in range(pages(ctx[b])):
                stack[top] = table[b, p]
                top += 1
    lens, offsets, t = [], [0], 0
    for b in range(B):
        end = ctx[b] + new[b] if new[b] >= 0 else 0
        if new[b] >= 0:
            for p in range(pages(ctx[b]), pages(end)):
                top -= 1
                table[b, p] = stack[top]
            for pos in range(ctx[b], end):
                slot = int(table[b, pos // page]) * page + pos % page
                slots[t] = slot if table[b, pos // page] >= 0 and slot < 2 ** 31 else -1
                positions[t] = pos
                t += 1
        lens.append(end)
        offsets.append(t)
    return {"table": table, "stack": stack, "lens": np.array(lens), "offsets": np.array(offsets), "slots": slots,
            "positions": positions, "left": top, "status": OK}


def round_code(y):
    """R: nearest even at 4 significant bits, below 2^-6 cut to a multiple of 2^-9, at most 448."""
    y = np.asarray(y, dtype=np.float64)
    a = np.where(np.isfinite(y), np.abs(y), 0.0)
    _, e = np.frexp(a)                       # a = m 2^e, m in [0.5, 1)
    step = np.ldexp(1.0, e - 4)
    r = np.rint(a / step) * step
    r = np.where(r < 2.0 ** -6, np.floor(r * 512) / 512, r)
    r = np.copysign(np.minimum(r, 448.0), y)
    return np.where(np.isfinite(y), r, np.nan)


def exponent(x):
    """The smallest e in [-64, 64] with |x| <= 448 * 2^e for every finite entry of the vector x."""
    a = np.max(np.where(np.isfinite(x), np.abs(x), 0.0), initial=0.0)
    e = E_MIN
    while e < E_MAX and a > 448.0 * 2.0 ** e:
        e += 1
    return e


class Cache:
    """Code values (fp64) and exponents of one pool, [pages, page, heads, dim] and [pages, heads]."""

    def __init__(self, codes, scales):
        self.value = e4m3_to_f64(np.asarray(codes, np.uint8)).reshape(np.shape(codes))
        self.scale = np.asarray(scales, np.float64).copy()

    def append(self, x_bits, slots):
        """Rows x_bits [T, heads, dim] (bf16 bits) to their slots, one token after the other."""
        x = bf16_to_f64(np.asarray(x_bits, np.uint16)).reshape(np.shape(x_bits))
        page = self.value.shape[1]
        for row, slot in zip(x, slots):
            slot = int(slot)
            if slot < 0 or slot >= self.value.shape[0] * page:
                continue
            p, off = divmod(slot, page)
            for h in range(x.shape[1]):
                e = exponent(row[h])
                if off:
                    old = int(np.log2(self.scale[p, h]))
                    if e > old:
                        self.value[p, :off, h] = round_code(self.value[p, :off, h] * 2.0 ** (old - e))
                    e = max(e, old)
                self.scale[p, h] = 2.0 ** e
                self.value[p, off, h] = round_code(row[h] / 2.0 ** e)

    def dequantised(self):
        return self.value * self.scale[:, None, :, None]


def paged_attention(Q_bits, K, V, table, lens, scale, window=0, v_scale=None):
    """Q_bits [B, Hq, D] (bf16 bits), K, V fp64 [pages, page, heads, D] (dequantised).  Returns O,
    lse and, for error bounds with normalised weights w_j: sum_j w_j |v_j| [B, Hq, D], max_j sum_d
    |q_d k_jd| [B, Hq], and what weights too small to be held can amount to [B, Hq]: 2^-40 of the
    largest w_j v_scale_j times 448 for each position (v_scale [pages, heads], 1 if not given), and
    2^-126 max |v|."""
    Q = bf16_to_f64(np.asarray(Q_bits, np.uint16)).reshape(np.shape(Q_bits))
    B, Hq, D = Q.shape
    page, heads = K.shape[1], K.shape[2]
    O, lse = np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf)
    spread, mass, floor = np.zeros((B, Hq, D)), np.zeros((B, Hq)), np.zeros((B, Hq))
    sc = float(np.float32(scale))
    for b in range(B):
        n = int(lens[b])
        pos = np.arange(max(0, n - window) if window else 0, n)
        if pos.size == 0:
            continue
        p, i = np.asarray(table)[b, pos // page], pos % page
        for h in range(Hq):
            kv = h // (Hq // heads)
            k, v = K[p, i, kv], V[p, i, kv]
            s = sc * (k @ Q[b, h])
            m = s.max()
            w = np.exp(s - m)
            O[b, h] = w @ v / w.sum()
            lse[b, h] = m + np.log(w.sum())
            spread[b, h] = w @ np.abs(v) / w.sum()
            mass[b, h] = np.max(np.abs(k) @ np.abs(Q[b, h]))
            sv = 1.0 if v_scale is None else np.asarray(v_scale, np.float64)[p, kv]
            floor[b, h] = pos.size * (2.0 ** -40 * 448 * np.max(w * sv) / w.sum() + 2.0 ** -126 * np.abs(v).max())
    return O, lse, spread, mass, floor
