"""The sampler's sums in two floats and its search for the bin in which a running sum reaches a border, compiled for the host: the same
code as on the GPU, in a block's threads one after the other."""
import ctypes
import shutil
import subprocess
from pathlib import Path

import numpy as np
import pytest

CSRC = Path(__file__).resolve().parents[1] / "gqa_attention_learned_head_gb300" / "csrc"

# A block's scan as the kernel makes it: each thread's sum, the lanes below it by doubling steps, the warps below it in order.
BLOCK = r"""
#include "sample_sums.h"
using namespace sinkattn;
constexpr int kThreads = 256, kEach = 4, kBins = kThreads * kEach;

template <typename Sum>
void scan(const Sum (&w)[kBins], Sum base, Sum (&before)[kThreads]) {
    Sum warps[kThreads / 32];
    for (int wp = 0; wp < kThreads / 32; ++wp) {
        Sum mine[32], incl[32];
        for (int l = 0; l < 32; ++l) {
            Sum m{};
            for (int i = 0; i < kEach; ++i) m = m + w[(wp * 32 + l) * kEach + i];
            mine[l] = incl[l] = m;
        }
        for (int o = 1; o < 32; o *= 2) {
            Sum old[32];
            for (int l = 0; l < 32; ++l) old[l] = incl[l];
            for (int l = o; l < 32; ++l) incl[l] = old[l] + old[l - o];
        }
        Sum below{};
        for (int v = 0; v < wp; ++v) below = below + warps[v];
        for (int l = 0; l < 32; ++l) before[wp * 32 + l] = base + (below + (l ? incl[l - 1] : Sum{}));
        warps[wp] = incl[30] + mine[31];
    }
}

// order: the threads as they come.  Answers: the bin, the sum before it, and how many bins begin below the goal and end
// at it or above.
template <typename Sum>
void search(const Sum (&w)[kBins], const unsigned* n, Sum base, Sum goal, const int* order, int* bin, Sum* at, int* claims) {
    Sum before[kThreads];
    scan(w, base, before);
    *bin = kBins;
    *claims = 0;
    for (int j = 0; j < kThreads; ++j) {
        const int t = order[j];
        Sum b = before[t], mine[kEach];
        unsigned here[kEach];
        for (int i = 0; i < kEach; ++i) mine[i] = w[t * kEach + i], here[i] = n[t * kEach + i];
        Sum c = b;
        for (int i = 0; i < kEach; ++i) {
            const Sum next = c + mine[i];
            if (c < goal && !(next < goal) && here[i]) ++*claims;
            c = next;
        }
        const int found = first_reaching(b, mine, here, goal, t * kEach, kBins);
        if (found < *bin) *bin = found, *at = b;
    }
}

extern "C" {
void search_f32(const float* w, const unsigned* n, float goal, const int* order, int* bin, float* at, int* claims) {
    float ww[kBins];
    for (int i = 0; i < kBins; ++i) ww[i] = w[i];
    search<float>(ww, n, 0.f, goal, order, bin, at, claims);
}
void search_pair(const float* w, const unsigned* n, const float* base, const float* goal, const int* order, int* bin, float* at, int* claims) {
    Pair ww[kBins], b;
    for (int i = 0; i < kBins; ++i) ww[i] = Pair{w[2 * i], w[2 * i + 1]};
    search<Pair>(ww, n, Pair{base[0], base[1]}, Pair{goal[0], goal[1]}, order, bin, &b, claims);
    at[0] = b.h, at[1] = b.l;
}
// The sums on both sides of each border between threads: behind the last bin of the one below, and before the first of the next.
void borders_f32(const float* w, float* sides) {
    float ww[kBins], before[kThreads];
    for (int i = 0; i < kBins; ++i) ww[i] = w[i];
    scan(ww, 0.f, before);
    for (int t = 0; t + 1 < kThreads; ++t) {
        float c = before[t];
        for (int i = 0; i < kEach; ++i) c = c + ww[t * kEach + i];
        sides[2 * t] = c, sides[2 * t + 1] = before[t + 1];
    }
}
void borders_pair(const float* w, const float* base, float* sides) {
    Pair ww[kBins], before[kThreads];
    for (int i = 0; i < kBins; ++i) ww[i] = Pair{w[2 * i], w[2 * i + 1]};
    scan(ww, Pair{base[0], base[1]}, before);
    for (int t = 0; t + 1 < kThreads; ++t) {
        Pair c = before[t];
        for (int i = 0; i < kEach; ++i) c = c + ww[t * kEach + i];
        sides[4 * t] = c.h, sides[4 * t + 1] = c.l, sides[4 * t + 2] = before[t + 1].h, sides[4 * t + 3] = before[t + 1].l;
    }
}
void add_pairs(const float* a, const float* b, float* out, int n) {
    for (int i = 0; i < n; ++i) {
        const Pair s = Pair{a[2 * i], a[2 * i + 1]} + Pair{b[2 * i], b[2 * i + 1]};
        out[2 * i] = s.h, out[2 * i + 1] = s.l;
    }
}
void times_count(const float* a, const unsigned* k, float* out, int n) {
    for (int i = 0; i < n; ++i) {
        const Pair s = times(Pair{a[2 * i], a[2 * i + 1]}, k[i]);
        out[2 * i] = s.h, out[2 * i + 1] = s.l;
    }
}
}
"""

BINS, THREADS = 1024, 256


def compile_host(tmp, text):
    """A shared library of C++ text that includes the kernels' headers: every product and sum rounded by itself."""
    src, lib = tmp / "host.cpp", tmp / "host.so"
    src.write_text(text)
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host compiler")
    subprocess.run([gxx, "-std=c++17", "-O2", "-ffp-contract=off", "-fPIC", "-shared", "-I", str(CSRC), str(src), "-o", str(lib)], check=True)
    return ctypes.CDLL(str(lib))


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    return compile_host(tmp_path_factory.mktemp("sums"), BLOCK)


def at(a):
    return a.ctypes.data_as(ctypes.c_void_p)


def pairs(x):
    """64-bit numbers as two floats each."""
    h = x.astype(np.float32)
    return np.ascontiguousarray(np.stack([h, (x - h).astype(np.float32)], -1))


def weights(gen):
    """Counts that fall with the bin, some bins empty, times the bin's weight."""
    n = gen.poisson(np.exp(gen.uniform(0, 6) - 0.004 * np.arange(BINS))).astype(np.uint32)
    return n, n * np.exp2(-(np.arange(BINS) + 0.5) / 32)


def answers(call, w, n, goal, kind):
    got = set()
    for order in (np.arange(THREADS), np.arange(THREADS)[::-1], np.random.default_rng(1).permutation(THREADS)):
        order = np.ascontiguousarray(order, dtype=np.int32)
        b, c, a = ctypes.c_int(), ctypes.c_int(), np.zeros(2, np.float32)
        call(order, ctypes.byref(b), at(a), ctypes.byref(c))
        got.add((b.value, a.tobytes(), c.value))
    assert len(got) == 1, (kind, got)  # the same bin, whoever comes first
    (found, mass, claims), = got
    return found, np.frombuffer(mass, np.float32), claims


@pytest.mark.parametrize("kind", ["f32", "pair"])
def test_one_bin_whoever_answers_first(host, kind):
    """Goals set between the two roundings of a thread's border: two threads hold a bin that begins below and ends at it or above, or
    none does."""
    gen = np.random.default_rng(7)
    none, two, across = 0, 0, 0
    for _ in range(400):
        n, exact = weights(gen)
        if kind == "f32":
            w = exact.astype(np.float32)
            sides = np.zeros((THREADS - 1, 2), np.float32)
            host.borders_f32(at(w), at(sides))
        else:
            w, base = pairs(exact * (1 + gen.random(BINS))), pairs(np.array(gen.uniform(0, 1e4)))
            sides = np.zeros((THREADS - 1, 2, 2), np.float32)
            host.borders_pair(at(w), at(base), at(sides))
        value = sides.astype(np.float64).reshape(THREADS - 1, 2, -1).sum(-1)
        apart = np.flatnonzero(value[:, 0] != value[:, 1])
        if not len(apart):
            continue
        at_warp = apart[apart % 32 == 31]
        for t in list(gen.choice(apart, 2)) + list(at_warp[:2]):
            goal = np.ascontiguousarray(sides[t, int(np.argmax(value[t]))])  # at the larger side, above the smaller
            if kind == "f32":
                call = lambda o, b, a, c: host.search_f32(at(w), at(n), ctypes.c_float(float(goal[0])), at(o), b, a, c)  # noqa: E731
            else:
                call = lambda o, b, a, c: host.search_pair(at(w), at(n), at(base), at(goal), at(o), b, a, c)  # noqa: E731
            found, mass, claims = answers(call, w, n, goal, kind)
            none += claims == 0
            two += claims == 2
            across += claims == 2 and t % 32 == 31
            assert found < BINS and n[found] > 0
            # the bin next to that border, or one whose sum is as near to it as the roundings are
            total = np.abs(value).max()
            behind = mass.astype(np.float64).sum() + np.asarray(w[found], dtype=np.float64).sum()
            goal64 = float(np.asarray(goal, np.float64).sum())
            near = total * (2.0**-20 if kind == "f32" else 2.0**-40)
            assert mass.astype(np.float64).sum() <= goal64 + near and behind >= goal64 - near
    assert none > 20 and two > 20 and across > 5, (none, two, across)  # (the case is met)


def test_a_goal_above_all_has_no_bin(host):
    n, w = weights(np.random.default_rng(3))
    w = w.astype(np.float32)
    call = lambda o, b, a, c: host.search_f32(at(w), at(n), ctypes.c_float(2 * float(w.sum())), at(o), b, a, c)  # noqa: E731
    assert answers(call, w, n, None, "f32")[0] == BINS


def test_sums_in_two_floats(host):
    """A sum of two pairs keeps 2^-46 of itself, a product with a count 2^-45 (two products of 2^-47 each and their sum)."""
    gen = np.random.default_rng(5)
    k = 20000
    a, b = (gen.random(k) * np.exp2(gen.integers(-40, 40, k)) for _ in range(2))
    out, (pa, pb) = np.zeros((k, 2), np.float32), (pairs(a), pairs(b))
    wide = lambda p: p.astype(np.longdouble).sum(-1)  # noqa: E731
    host.add_pairs(at(pa), at(pb), at(out), k)
    want = wide(pa) + wide(pb)
    assert np.all(np.abs(wide(out) - want) <= want * 2.0**-46)
    count = gen.integers(0, 2**30, k).astype(np.uint32)
    host.times_count(at(pa), at(count), at(out), k)
    want = wide(pa) * count
    assert np.all(np.abs(wide(out) - want) <= want * 2.0**-45)
