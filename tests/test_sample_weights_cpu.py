"""The sampler's weights in two floats, compiled for the host: every 16-bit logit beside a much larger one, 32-bit logits, temperatures
and sizes far out.

Bound of a weight's error, 2^-28.5 of itself: with y = k / 32 + r, |r| <= 2^-6, r has two roundings of half a step of numbers below 2^-6
(2^-31 each, times ln 2), the polynomial (0.69, half a step 2^-25) times r, its product with r (below 2^-6: 2^-31), the weight's part
with r (below 2^-5 of a root below 2, so 2^-30.5 of the weight at most): (2 ln 2 + 1 + 1 + 1.42) 2^-31 = 2^-28.7.
ch + cl is log2(e) / t to 2^-48, which at |y| <= 4206 is 2^-36 of the weight."""
import numpy as np
import pytest
import torch

from test_sample_sums_cpu import at, compile_host

CODE = r"""
#include "sample_weights.h"
using namespace sinkattn;
static const float roots[32][2] = SINKATTN_ROOTS;

extern "C" void weights(const float* z, int n, float m, float t, float* out, double* row) {
    const RowScale g = row_scale(m, t);
    row[0] = g.ref, row[1] = g.base;
    for (int i = 0; i < n; ++i) {
        float y, k, r, h, l;
        split_power<OneByOne>(g, z[i], y, k, r);
        union { float f; int i; } bits{k};
        const int n2 = bits.i - 0x4B400000;
        root_times_power<OneByOne>(roots[n2 & 31][0], roots[n2 & 31][1], r, h, l);
        const bool in = y > g.least;
        out[2 * i] = in ? std::ldexp(h, (n2 >> 5) - g.base) : 0.f;
        out[2 * i + 1] = in ? std::ldexp(l, (n2 >> 5) - g.base) : 0.f;
    }
}
"""
BOUND = 2.0**-28.5


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    return compile_host(tmp_path_factory.mktemp("weights"), CODE)


def check(host, z, m, t):
    """z float32 logits up to m."""
    z = np.ascontiguousarray(z, dtype=np.float32)
    out, row = np.zeros((len(z), 2), np.float32), np.zeros(2)
    host.weights(at(z), len(z), np.ctypeslib.ctypes.c_float(m), np.ctypeslib.ctypes.c_float(t), at(out), at(row))
    m, t = np.longdouble(np.float32(m)), np.longdouble(np.float32(t))
    wide = out.astype(np.longdouble).sum(-1)
    x = (z.astype(np.longdouble) - m) / t
    with np.errstate(over="ignore"):
        want = np.exp2((z.astype(np.longdouble) - np.longdouble(row[0])) / t / np.log(np.longdouble(2)) - np.longdouble(row[1]))
    has = x > -109 * np.log(np.longdouble(2))
    off = np.abs(wide - want)[has] / want[has]
    assert off.max() <= BOUND, float(np.log2(off.max()))
    assert row[0] in (0.0, m) and 1 - 2.0**-11 <= wide[np.argmax(z)] < 2 + 2.0**-11  # (y is rounded before it gives the base)
    assert np.all(wide[x < -112 * np.log(np.longdouble(2))] == 0)
    assert np.all(np.abs(out[:, 1]) <= 2.0**-24 * out[:, 0])
    return off


def sixteen(dtype):
    z = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(dtype).float().numpy()
    return z[np.isfinite(z)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("m,t", [(20.0, 1.0), (20.0, 5.0), (100.0, 100.0), (1.5, 0.7), (0.0, 1.0), (-3.25, 0.31), (-2e-4, 1e-4), (20.0, 0.007),
                                 (-60.0, 0.02), (3e4, 1.0), (6e4, 1e4)])
def test_every_16_bit_logit(host, dtype, m, t):
    z = sixteen(dtype)
    m = float(torch.tensor(m).to(dtype))
    check(host, z[z <= m], m, t)


@pytest.mark.parametrize("seed", range(40))
def test_32_bit_logits(host, seed):
    gen = np.random.default_rng(seed)
    t = np.float32(np.exp2(gen.uniform(-30, 30)))
    m = np.float32(gen.choice([0.0, 1.0, -1.0, 50.0, 3000.0, -2800.0, 2.0**20]) * t * gen.uniform(0.3, 1))
    x = np.concatenate([gen.uniform(-75, 0, 4000), -np.exp2(gen.uniform(-40, 6, 4000)), [0.0]])
    z = np.minimum((np.float64(m) + x * np.float64(t)).astype(np.float32), m)
    off = check(host, np.concatenate([z, np.minimum(np.float32(1e-4) * gen.standard_normal(100).astype(np.float32), m)]), m, t)
    assert off.size > 4000


def test_masked_and_far_logits(host):
    low = np.finfo(np.float32).min
    for m, t in ((5.0, 1.0), (1e30, 1e-20), (5.0, 1e-38), (low, 1.0)):
        z = np.array([m, low, -1e30, -np.inf], np.float32)
        check(host, z[z <= np.float32(m)], m, t)  # (m is the largest)


def test_one_temperature_for_all(host):
    """An infinite one: all finite logits weigh the same."""
    out, row, z = np.zeros((4, 2), np.float32), np.zeros(2), np.array([3e38, 1.0, -3e38, -np.inf], np.float32)
    host.weights(at(z), 4, np.ctypeslib.ctypes.c_float(3e38), np.ctypeslib.ctypes.c_float(np.inf), at(out), at(row))
    assert out[:3, 0].tolist() == [1.0] * 3 and out[3, 0] == 0 and not out[:, 1].any() and row[1] == 0
