"""Places of the paged 8-bit cache that are written again: draft tokens that were rejected."""
import numpy as np
import pytest
import torch

import invariant_deterministic_gemm_bi_b200 as bg
from tests.test_gpu_kv_cache import fresh, ints, prompt_slots, tokens, write_and_compare

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("heads,dim", [(2, 128), (3, 64)])
def test_a_discarded_token_keeps_its_exponent_until_the_page_starts_anew(page, heads, dim):
    kept, draft, after = page // 2 + 3, 4, 3
    cache = fresh(2, page, heads, dim)
    K, V = tokens(kept + after, heads, dim, 201, 0.5), tokens(kept + after, heads, dim, 202, 0.5)
    K2, V2 = tokens(draft, heads, dim, 203, 0.5) * 64, tokens(draft, heads, dim, 204, 0.5) * 64
    write_and_compare(cache, K[:kept], V[:kept], prompt_slots([1], 0, kept, page))
    write_and_compare(cache, K2, V2, prompt_slots([1], kept, draft, page))
    # the final tokens over the draft's places: as the oracle, which joins what the scale has seen
    write_and_compare(cache, K[kept:], V[kept:], prompt_slots([1], kept, after, page))
    n = kept + after
    alone = fresh(2, page, heads, dim)
    slots = prompt_slots([1], 0, n, page)
    write_and_compare(alone, K, V, slots)
    assert torch.all(cache.k_scale[1] > alone.k_scale[1]) and torch.all(cache.v_scale[1] > alone.v_scale[1])
    assert not torch.equal(cache.k[1, :n], alone.k[1, :n])
    # the page from its first place: the final tokens' own
    bg.bi_kv_append_e4m3(cache, K, V, ints(slots))
    assert torch.equal(cache.k[1, :n], alone.k[1, :n]) and torch.equal(cache.v[1, :n], alone.v[1, :n])
    assert torch.equal(cache.k_scale[1], alone.k_scale[1]) and torch.equal(cache.v_scale[1], alone.v_scale[1])


def test_a_draft_that_needed_a_page_of_its_own():
    # the draft's tokens in a new page are gone with the next first place; those in the old one are not
    page, heads, dim = 16, 1, 64
    K, V = tokens(20, heads, dim, 211, 0.5), tokens(20, heads, dim, 212, 0.5)
    big = tokens(6, heads, dim, 213, 0.5) * 64
    cache, alone = fresh(2, page, heads, dim), fresh(2, page, heads, dim)
    write_and_compare(cache, K[:16], V[:16], prompt_slots([0, 1], 0, 16, page))
    write_and_compare(cache, big, big, prompt_slots([0, 1], 16, 6, page))
    write_and_compare(cache, K[16:], V[16:], prompt_slots([0, 1], 16, 4, page))
    write_and_compare(alone, K, V, prompt_slots([0, 1], 0, 20, page))
    for a, b in ((cache.k, alone.k), (cache.v, alone.v)):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1, :4], b[1, :4])
    assert torch.equal(cache.k_scale, alone.k_scale) and torch.equal(cache.v_scale, alone.v_scale)
