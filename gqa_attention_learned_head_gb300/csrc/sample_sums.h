// sample_sums.h -- sums in two floats, and where a running sum reaches a border: what sample.cu compares when it cuts a row's weights.
// Plain arithmetic without CUDA's types, so that the same code also compiles for the host (without contraction of products and sums).
#pragma once
#include <cmath>

#ifdef __CUDACC__
#define SINKATTN_HD __host__ __device__ __forceinline__
#else
#define SINKATTN_HD inline
#endif

namespace sinkattn {

// A product rounded by itself.
SINKATTN_HD float product(float a, float b) {
#ifdef __CUDA_ARCH__
    return __fmul_rn(a, b);
#else
    return a * b;
#endif
}

// A sum as h + l, |l| at most half a step of h: about 46 bits.  (64-bit arithmetic runs at 1/64 of the 32-bit rate on this GPU; this
// takes some ten 32-bit instructions.)
struct Pair {
    float h, l;
};
SINKATTN_HD Pair operator+(Pair a, Pair b) {
    const float s = a.h + b.h, t = s - a.h;
    const float e = ((a.h - (s - t)) + (b.h - t)) + (a.l + b.l);
    const float h = s + e;
    return {h, e - (h - s)};
}
SINKATTN_HD Pair times(Pair a, float x) {
    const float p = product(a.h, x), e = fmaf(a.h, x, -p) + product(a.l, x);
    const float h = p + e;
    return {h, e - (h - p)};
}
SINKATTN_HD Pair times(Pair a, unsigned n) {  // (both parts of n are exact in f32)
    return times(a, (float)(n & ~0xFFFu)) + times(a, (float)(n & 0xFFFu));
}
SINKATTN_HD bool operator<(Pair a, Pair b) { return a.h < b.h || (a.h == b.h && a.l < b.l); }

// The first of a thread's kEach bins, number `first` and up, that is not empty and at whose end the running sum is no longer below
// `goal`; `none` where there is none.  b: the sum before the first bin, then the one before the bin found.
// Threads' sums before them come from a scan and are other roundings than the sum behind the thread below: asked for the one bin that
// begins below the goal and ends at it or above, two threads or none may answer.  The lowest of the answers to this question is one
// bin, whoever answers first.
template <int kEach, typename Sum>
SINKATTN_HD int first_reaching(Sum& b, const Sum (&w)[kEach], const unsigned (&n)[kEach], Sum goal, int first, int none) {
    for (int i = 0; i < kEach; ++i) {
        const Sum next = b + w[i];
        if (n[i] && !(next < goal)) return first + i;
        b = next;
    }
    return none;
}

}  // namespace sinkattn
