// sample_weights.h -- a logit's weight e^((z - m) / t) in two floats, but for one factor that a row's weights share.
// Written for one logit or for two at once (O: the operations); the same code compiles for the host (without contraction of products
// and sums).
//
// With ch + cl = log2(e) / t in two floats a weight is 2^y, y = d (ch + cl), over 2^base.  d is the logit itself where m log2(e) / t is
// within kNear: its low bits would be lost in z - m (bf16 or f16 logits of 1e-4 beside one of 20, as much as 2^-20 of their
// weight).  Else it is z - m, which is exact for all logits that have a weight: those are within 3% of m.  Then
//     k = rint(32 y),  r = y - k / 32,  2^y = 2^(k / 32) (1 + r c1 + r^2 c2 + ..),  |r| at most 1/64.
// Roundings: r's two (each 2^-31 in y), the polynomial's, that of its product with r and of r's part of the weight (each 2^-31 of the
// weight, or 2^-30.5): off by at most 2^-28.5 of the weight, alike for logits of the same value.  What cl and the polynomial leave
// out is below 2^-36.
#pragma once
#include "sample_sums.h"

namespace sinkattn {

constexpr float kNear = 4096.f;    // the largest |m log2(e) / t| at which d is the logit itself
constexpr float kFloor = 110.f;    // a weight below 2^-110 of the largest is nothing
constexpr float kLargestScale = 3e38f;

struct RowScale {
    float ref;     // d = z - ref: 0 or the largest logit
    float ch, cl;  // log2(e) / t in two floats
    float least;   // weights are of y above this one
    int base;      // weights are 2^(y - base), of the largest logit from 1 to 2
};
// m the largest logit, t > 0.
SINKATTN_HD RowScale row_scale(float m, float t) {
    constexpr float kLog2eH = 1.442695f, kLog2eL = 1.925963033500927e-08f;  // (their sum is log2(e) to 2^-49)
    RowScale g;
    g.ch = kLog2eH / t;
    g.cl = (fmaf(-g.ch, t, kLog2eH) + kLog2eL) / t;
    const bool tiny = !(g.ch < kLargestScale);
    if (tiny) g.ch = kLargestScale, g.cl = 0.f;               // a temperature so small that only the largest logits count
    if (!(t < __builtin_huge_valf())) g.ch = g.cl = 0.f;      // one so large that all count alike
    const float y = product(m, g.ch);
    const bool near = !tiny && y >= -kNear && y <= kNear;
    g.ref = near ? 0.f : m;
    g.base = near ? (int)floorf(y) : 0;
    g.least = (near ? y : 0.f) - kFloor;
    return g;
}
// One number at a time (on the GPU: two, sample.cu).
struct OneByOne {
    using F = float;
    static SINKATTN_HD F all(float x) { return x; }
    static SINKATTN_HD F add(F a, F b) { return a + b; }
    static SINKATTN_HD F mul(F a, F b) { return product(a, b); }
    static SINKATTN_HD F fma(F a, F b, F c) { return fmaf(a, b, c); }
};

// y, rounded, k + 1.5 * 2^23 and r of a logit.
template <typename O, typename F = typename O::F>
SINKATTN_HD void split_power(const RowScale& g, F z, F& y, F& k, F& r) {
    constexpr float kMagic = 12582912.f;  // 1.5 * 2^23
    const F d = O::add(z, O::all(-g.ref));
    y = O::mul(d, O::all(g.ch));
    k = O::fma(y, O::all(32.f), O::all(kMagic));
    const F part = O::mul(O::add(k, O::all(-kMagic)), O::all(-1.f / 32.f));
    r = O::fma(d, O::all(g.cl), O::fma(d, O::all(g.ch), part));
}
// (h, l) = (th + tl) 2^r, |l| at most half a step of h; th + tl the table's entry.
template <typename O, typename F = typename O::F>
SINKATTN_HD void root_times_power(F th, F tl, F r, F& h, F& l) {
    // 2^r - 1 = r (ln 2 + r (ln 2^2 / 2 + r (ln 2^3 / 6 + r ln 2^4 / 24))), the next term below 2^-39
    F q = O::fma(r, O::all(0.00961812911f), O::all(0.0555041087f));
    q = O::fma(r, q, O::all(0.240226507f));
    q = O::fma(r, q, O::all(0.693147181f));
    const F v = O::fma(th, O::mul(r, q), tl);
    h = O::add(th, v);
    l = O::add(v, O::fma(h, O::all(-1.f), th));
}

// 2^(i / 32) in two floats, from the definition to 60 digits.
#define SINKATTN_ROOTS                                                                                                            \
    {                                                                                                                             \
        {1.e+00f, 0.e+00f}, {1.0218972e+00f, -4.81156e-08f}, {1.0442737e+00f, 4.83347e-08f}, {1.0671405e+00f, -5.933752e-08f},    \
        {1.0905077e+00f, -1.307754e-08f}, {1.1143868e+00f, -5.43554e-08f}, {1.1387886e+00f, 5.3862223e-08f},                      \
        {1.1637249e+00f, -4.0514415e-08f}, {1.1892071e+00f, 3.7976353e-08f}, {1.2152474e+00f, -3.267395e-08f},                    \
        {1.2418578e+00f, 4.496838e-08f}, {1.269051e+00f, 1.4193333e-09f}, {1.2968396e+00f, -4.0189995e-08f},                      \
        {1.3252367e+00f, -3.4963733e-08f}, {1.3542556e+00f, -1.0123349e-08f}, {1.38391e+00f, -5.8755774e-08f},                    \
        {1.4142135e+00f, 2.4203235e-08f}, {1.4451808e+00f, 3.3242e-08f}, {1.4768262e+00f, -4.500899e-08f},                        \
        {1.5091645e+00f, -2.4959373e-08f}, {1.5422108e+00f, 8.070905e-09f}, {1.5759809e+00f, -5.6610254e-08f},                    \
        {1.6104903e+00f, 9.836217e-09f}, {1.6457555e+00f, -5.124972e-08f}, {1.6817929e+00f, -2.4755327e-08f},                     \
        {1.7186193e+00f, -4.8496176e-08f}, {1.7562522e+00f, -9.23577e-09f}, {1.7947091e+00f, -1.1415045e-08f},                    \
        {1.8340081e+00f, -1.1239278e-08f}, {1.8741677e+00f, -4.6630056e-08f}, {1.9152066e+00f, 9.845328e-09f},                    \
        {1.9571441e+00f, -1.7021804e-08f}                                                                                        \
    }

}  // namespace sinkattn
