"""The decode over the cache held in 8 bits where pages' value scales lie far apart: one value of one token far above all others, so that its
page's other dimensions hold nothing, at like scores; and large values at scores far below.  Every dimension is checked by itself."""
import numpy as np
import pytest
import torch

import oracle
import q8_reference as R
from gqa_attention_learned_head_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S():
    from gqa_attention_learned_head_gb300 import sinkattn

    return sinkattn


def decode_and_check(S, d, cache, what, workers, score=1e-4):
    g = d.to("cuda")
    call = lambda v: oracle.decode(d.q, cache.k_wide, v, d.page_table, d.kv_lens, d.sinks, d.scale)  # noqa: E731
    (ro, rl), (spread, _) = call(cache.v_wide), call(cache.v_wide.abs())
    for w in workers:
        out, lse = S.sinkattn_decode_q8(g.q, *cache.args, g.page_table, g.kv_lens, g.sinks, g.scale, num_workers=w)
        assert S.sinkattn_get_error() == 0
        R.close_attention(out.float().cpu().numpy(), lse.cpu().numpy(), ro, rl, spread, f"{what}, {w} shares", score=score)


@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (16, 1), (5, 5)])
@pytest.mark.parametrize("gap", [3, 10, 20, 30, 40, 60, 79])
def test_one_value_far_above(S, Hq, Hkv, gap):
    """In the first, a middle, the last page of a request, in every other page, and in two sizes."""
    lens = [400, 37, 1333, 90, 16, 160]
    d = W.make_decode(len(lens), Hq, Hkv, lens, seed=gap)
    v = d.v_pages.float() * 2.0**-33
    at = lambda b, j: int(d.page_table[b, j])  # noqa: E731
    big = 3 * 2.0 ** (gap - 33)
    for page, factor in [(at(0, 0), 1), (at(1, 2), 1), (at(2, 40), 1), (at(3, 1), -1), (at(3, 4), 2.0 ** -(gap // 2)), (at(4, 0), 1)] + [
            (at(5, j), 1) for j in range(0, 10, 2)]:
        v[page, :, 3, 11] = big * factor
    decode_and_check(S, d, R.Cache(0.1 * d.k_pages.float(), v), f"gap {gap}", (1, 0, 7, 64))


@pytest.mark.parametrize("Hkv", [2, 9])
@pytest.mark.parametrize("gap,below", [(20, 3.0), (40, 3.0), (60, 5.0), (60, 3.0), (79, 6.0), (79, 2.0)])
def test_large_values_far_below(S, Hkv, gap, below):
    """Scores `below` x 6.4 under the others' (some 9 bits each), values 2^gap above: they are most of the output or next to nothing."""
    lens = [400, 37, 800, 64]
    d = W.make_decode(len(lens), Hkv, Hkv, lens, seed=gap)
    k, v = 0.1 * d.k_pages.float(), d.v_pages.float() * 2.0**-33
    for b, pages in enumerate(([3, 20], [0], [0, 1, 2, 30, 49], [3])):
        for j in pages:
            p = int(d.page_table[b, j])
            k[p] = -below * d.q[b].float().sign()[:, None, :]
            v[p] *= 2.0**gap
    # |q k| sums to 6.4 x below instead of 5
    decode_and_check(S, d, R.Cache(k, v), f"gap {gap}, {below}", (1, 0, 7), score=1e-4 * max(1.0, 6.4 * below / 5))


def test_scales_that_wander(S):
    """Each page's scale some powers of two from the last one's, up and down over the whole range."""
    lens = [3000, 1000]
    d = W.make_decode(2, 16, 2, lens, seed=8)
    gen = np.random.default_rng(8)
    v = d.v_pages.float()
    for b in range(2):
        e = 0
        for j in range((lens[b] + 15) // 16):
            e = int(np.clip(e + gen.integers(-6, 7), -31, 31))
            v[int(d.page_table[b, j])] *= 2.0**e
    decode_and_check(S, d, R.Cache(d.k_pages.float(), v), "wandering", (1, 0, 5))
