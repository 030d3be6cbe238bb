"""Sampling where many 16-bit logits share one value next to zero beside a far larger one, so that z - m loses their low bits: random
numbers next to tokens' borders pick the tokens that exact arithmetic picks."""
import numpy as np
import pytest
import torch

from test_sample_gpu import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S():
    from gqa_attention_learned_head_gb300 import sinkattn

    return sinkattn


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("m,t", [(20.0, 5.0), (20.0, 2.0), (100.0, 30.0)])
def test_ties_next_to_zero(S, dtype, m, t):
    gen = np.random.default_rng(int(m + t))
    V, N = 60000, 48
    value = 218 * 2.0**-21  # (both types hold it; z - m lies half a step of 32 bits from the next number at m = 20, 3/8 at 100)
    z = np.where(gen.random(V) < 0.5, value, gen.choice([0.5, -0.25, 1.0, -2.0], V))
    z[gen.integers(0, V)] = m
    w = np.exp((z - m) / t)
    line = np.cumsum(w) / w.sum()
    u = gen.random(1 << 20).astype(np.float32)
    i = np.searchsorted(line, u)
    near = np.minimum(np.abs(line[np.minimum(i, V - 1)] - u), np.abs(line[np.maximum(i - 1, 0)] - u))
    # a weight is off by at most 2^-28.5, the sum up to a border as a share of all by half of that (the errors of the two groups of
    # tokens work against each other, by s (1 - s) 2^-28.5 2 at most)
    u = u[(near > 2.0**-28) & (near < 2.0**-25)][:N]
    assert len(u) == N
    logits = torch.from_numpy(z).to(dtype).cuda().expand(N, V).contiguous()
    check(S, logits, u, [t] * N)
