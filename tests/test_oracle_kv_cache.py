"""Pins of the paged cache's oracle: hand-worked tables, the rounding against exact rationals, the
write's independence of how tokens are grouped, and attention against a dense closed form."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from invariant_deterministic_gemm_bi_b200 import inputs
from oracle import kv_cache as okv
from oracle.oracle import e4m3_to_f64

E4M3 = sorted({abs(float(v)) for v in e4m3_to_f64(np.arange(256, dtype=np.uint8)) if np.isfinite(v)})


def test_block_tables_by_hand():
    # pages of 16: request 0 has 20 tokens in pages 7, 3 and gets 13 (one more page); request 1 ends
    # and gives back 5; request 2 is new with 17 tokens; request 3 stays as it is
    table = np.full((4, 4), -9)
    table[0, :2] = [7, 3]
    table[1, :1] = [5]
    table[3, :1] = [1]
    got = okv.block_tables([20, 9, 0, 3], [13, -1, 17, 0], 16, [2, 4, 6, 8, -1], 4, table, 32)
    assert got["status"] == 0
    # 5 is pushed, then popped for request 0; request 2 gets 8 and 6
    assert got["table"].tolist() == [[7, 3, 5, -9], [5, -9, -9, -9], [8, 6, -9, -9], [1, -9, -9, -9]]
    assert got["stack"].tolist() == [2, 4, 6, 8, 5] and got["left"] == 2
    assert got["lens"].tolist() == [33, 0, 17, 3] and got["offsets"].tolist() == [0, 13, 13, 30, 30]
    want = [3 * 16 + i for i in range(4, 16)] + [5 * 16] + [8 * 16 + i for i in range(16)] + [6 * 16, -1, -1]
    assert got["slots"].tolist() == want
    assert got["positions"].tolist() == list(range(20, 33)) + list(range(17)) + [-1, -1]


@pytest.mark.parametrize("change,status", [
    ({"ctx": [-1, 0]}, 1), ({"new": [-2, 0]}, 1), ({"count": 9}, 1), ({"count": -1}, 1),
    ({"new": [49, 0]}, 3), ({"new": [17, 20]}, 3), ({"new": [33, 1], "count": 2}, 3),
    ({"new": [-1, 0], "count": 8, "ctx": [5, 0]}, 3)])
def test_block_tables_that_do_not_fit_change_nothing(change, status):
    a = {"ctx": [3, 0], "new": [1, 1], "count": 4} | change
    table = np.full((2, 3), 1)
    got = okv.block_tables(a["ctx"], a["new"], 16, np.arange(8), a["count"], table, 36)
    assert got["status"] == status and got["lens"].tolist() == a["ctx"] and got["left"] == a["count"]
    assert np.all(got["slots"] == -1) and np.array_equal(got["table"], table)
    assert np.array_equal(got["stack"], np.arange(8)) and np.all(got["offsets"] == 0)


def test_round_code_is_nearest_for_normals_and_a_cut_below():
    rng = np.random.default_rng(1)
    y = np.concatenate([rng.uniform(-448, 448, 500), rng.standard_normal(500), rng.standard_normal(800) * 2.0 ** -7,
                        [0.0, 2.0 ** -6, 2.0 ** -9, 2.0 ** -10, 0.99 * 2.0 ** -9, 464.0, 1e9]])
    for v, got in zip(y, okv.round_code(y)):
        a = Fraction(abs(float(v)))
        if a < Fraction(1, 64) and got < 2.0 ** -6:
            # the largest subnormal value at or below the value rounded to 4 bits
            assert abs(got) in E4M3 and abs(abs(got) - float(a)) < 2.0 ** -9
        elif a <= 448:
            near = min(abs(Fraction(e) - a) for e in E4M3)
            assert abs(got) in E4M3 and abs(Fraction(abs(float(got))) - a) == near
        else:
            assert abs(got) == 448.0
        assert np.signbit(got) == np.signbit(v)
    assert np.isnan(okv.round_code(np.array([np.nan, np.inf, -np.inf]))).all()
    # ties go to the even code
    assert okv.round_code(np.array([17.0, 19.0, 1.0625, 1.1875])).tolist() == [16.0, 20.0, 1.0, 1.25]


def test_round_code_composes():
    rng = np.random.default_rng(2)
    x = rng.standard_normal(20000) * 2.0 ** rng.integers(-14, 6, 20000)
    for d in range(0, 12):
        assert np.array_equal(okv.round_code(okv.round_code(x) * 2.0 ** -d), okv.round_code(x * 2.0 ** -d))


@pytest.mark.parametrize("amax,e", [(0.0, -64), (448.0, 0), (450.0, 1), (1.75, -8), (1.7578125, -7), (1e-30, -64),
                                    (3e38, 64), (896.0, 1)])
def test_exponents(amax, e):
    assert okv.exponent(np.array([amax, -amax / 2, np.inf, np.nan])) == e


def test_the_page_is_a_function_of_its_tokens():
    # tokens of growing magnitude, written one at a time (the oracle's way) against the definition
    # applied once with the final exponent
    g = np.random.default_rng(3)
    x = (g.standard_normal((16, 2, 64)) * 2.0 ** (np.arange(16)[:, None, None] - 9)).astype(np.float32)
    bits = inputs.to_numpy_bits(torch.from_numpy(x).to(torch.bfloat16))
    c = okv.Cache(np.full((3, 16, 2, 64), 0x7F), np.full((3, 2), 8.0))
    c.append(bits, np.arange(16, 32))
    xb = torch.from_numpy(x).to(torch.bfloat16).double().numpy()
    for h in range(2):
        e = okv.exponent(xb[:, h].ravel())
        assert c.scale[1, h] == 2.0 ** e
        assert np.array_equal(c.value[1, :, h], okv.round_code(xb[:, h] / 2.0 ** e))
    assert np.isnan(c.value[[0, 2]]).all() and np.all(c.scale[[0, 2]] == 8.0)


def test_a_place_written_again_joins_what_was_there():
    g = np.random.default_rng(5)
    x = torch.from_numpy(g.standard_normal((12, 1, 64)).astype(np.float32)).to(torch.bfloat16)
    x[8:] *= 64
    bits, xd = inputs.to_numpy_bits(x), x.double().numpy()
    c = okv.Cache(np.full((1, 16, 1, 64), 0x7F), np.full((1, 1), 8.0))
    c.append(bits, np.arange(12))
    c.append(bits[:2], np.array([8, 9]))             # two small tokens over the first large ones
    e = okv.exponent(xd.ravel())                     # that of all tokens the page has seen
    assert c.scale[0, 0] == 2.0 ** e and e > okv.exponent(xd[:8].ravel())
    assert np.array_equal(c.value[0, :10, 0], okv.round_code(np.concatenate([xd[:8], xd[:2]])[:, 0] / 2.0 ** e))
    c.append(bits[:8], np.arange(8))                 # from the first place: the page starts anew
    assert c.scale[0, 0] == 2.0 ** okv.exponent(xd[:8].ravel())


def test_popped_pages_stay_in_the_stacks_entries():
    # one page comes back and three go: the old top is 2, the new one 0, and the pushed page's entry keeps it
    table = np.array([[9, -1], [-1, -1], [-1, -1], [-1, -1]])
    got = okv.block_tables([3, 0, 0, 0], [-1, 1, 1, 1], 16, [4, 5, -7, -8], 2, table, 3)
    assert got["stack"].tolist() == [4, 5, 9, -8] and got["left"] == 0
    assert got["table"][1:, 0].tolist() == [9, 5, 4] and got["table"][0, 0] == 9


def test_attention_reads_the_paged_positions():
    g = np.random.default_rng(4)
    pages, page, heads, D, n = 9, 16, 2, 64, 50
    K, V = g.standard_normal((pages, page, heads, D)), g.standard_normal((pages, page, heads, D))
    table = np.array([[4, 0, 7, 2, 99]])
    Qb = inputs.to_numpy_bits(torch.from_numpy(g.standard_normal((1, 4, D))).to(torch.bfloat16))
    Q = torch.from_numpy(Qb.view(np.int16)).view(torch.bfloat16).double()
    O, lse, _, _, _ = okv.paged_attention(Qb, K, V, table, [n], 0.125, window=23)
    k = torch.from_numpy(K[table[0, :4]].reshape(-1, heads, D))[n - 23:n]
    v = torch.from_numpy(V[table[0, :4]].reshape(-1, heads, D))[n - 23:n]
    for h in range(4):
        s = 0.125 * k[:, h // 2] @ Q[0, h]
        assert np.allclose(O[0, h], (torch.softmax(s, 0) @ v[:, h // 2]).numpy(), rtol=1e-12)
        assert np.isclose(lse[0, h], torch.logsumexp(s, 0).item(), rtol=1e-12)
    O, lse, _, _, _ = okv.paged_attention(Qb, K, V, table, [0], 0.125)
    assert np.all(O == 0) and np.all(np.isneginf(lse))
