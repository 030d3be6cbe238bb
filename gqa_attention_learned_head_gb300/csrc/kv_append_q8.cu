// kv_append_q8.cu -- new tokens into a cache held in 8 bits: QKV bias and YaRN rotation (or ready keys and values), the scale of each
// page and head, and the codes.
//
// Sources: "GPT-OSS on day 0" (Perplexity), section "Attention: GQA with attention sinks" (bias, YaRN) and "Accelerating Sonar
// through speculation", section "Inference with speculative decoding" (slots of the next tokens in per-request pages).  The posts
// hold their cache in 16 bits; the 8-bit form is this library's.
//
// For a (page, KV head) whose slots a..b-1 the call writes, with x_t the new values (k: after bias and rotation) in 32 bits:
//     e_new = the smallest e with max |x| <= 448 * 2^e,   e = a > 0 ? max(e_old, e_new) : e_new        (within -40..40)
//     code_t = e4m3(x_t 2^-e),   and where e > e_old the codes of slots 0..a-1 become e4m3(code 2^(e_old - e)).
// One rounding from 32 bits to 8; the held tokens move exactly, but for those that become subnormal codes.
//
// HBM-bound elementwise work.  A page's scale needs all of its new tokens first, so the unit of work is a page of a sequence (its up
// to 16 new tokens), one CTA each, and a group of lanes keeps one head's tokens in registers from the load over the maximum to the
// store: each value is read once.  Four lanes take a (token, head), as in prologue.cu; a group is 4 x (tokens rounded up to a power of two) lanes, so that
// a decode step's single token keeps 8 heads of a warp busy and a full page 8 tokens twice.  Units are numbered without a scan of the
// lengths: sequence n's begin at (cu_seqlens[n] + 30 n) / 16, since its pages are at most (L + 30) / 16; the few numbers between are
// idle CTAs.
//
// Measured (GB300, 64 query and 8 KV heads, bias, rotation): eight chunks of 256 to 2048 tokens 39.6 us, 4.5 TB/s = 66% of the copy
// rate (CTAs of 8 warps 42.9; fewer registers, and with them more warps an SM, 51 to 61: what counts is the loads a warp has in flight,
// the next heads' while these are computed); 128 single tokens 4.4 us, the latency of one kernel.  Ready keys and values: 8.5 us (9113
// tokens, out of L2), 3.0 us.
#include "args_q8.h"
#include "ptx.cuh"
#include "q8.cuh"

namespace sinkattn {
namespace {

constexpr int kWarps = 4;
// Up to so many units (two for each of 152 SMs) their heads are dealt to two CTAs each.  Measured with one and with two, 64 query and 8 KV
// heads: chunks, 144 units 28.7 and 18.9 us, 306 units 31.9 and 24.4, 336 units 32.5 and 37.2, 516 units 37.4 and 40.9; single
// tokens (most units of which are idle) 249 units 4.8 and 4.3, 497 units 5.3 and 4.6, 621 units 5.4 and 5.8.
constexpr long long kFewUnits = 304;
constexpr float kInf = __builtin_huge_valf();

__device__ __forceinline__ float lo_bf16(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }

// The eight bf16 values of a 16-byte piece, in order, as floats.
__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = lo_bf16(w[i]);
        f[2 * i + 1] = hi_bf16(w[i]);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}

// The largest n in [0, N) whose first unit, (cu_seqlens[n] + 30 n) / 16, is at most u: 32 places a step, all lanes alike.
__device__ __forceinline__ int sequence_of(const int32_t* cu, int N, long long u, int lane) {
    int lo = 0, n = N;  // the answer is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int at = lo + lane * step;
        const bool in = lane * step < n && (((long long)__ldg(&cu[at]) + 30ll * at) >> 4) <= u;
        const unsigned yes = __ballot_sync(0xffffffffu, in);
        const int k = yes ? 31 - __clz(yes) : 0;
        lo += k * step;
        n = min(step, n - k * step);
    }
    return lo;
}

template <bool kPrologue, bool kInter>  // kInter: pairs (2d, 2d + 1) instead of (d, d + 32)
__global__ void __launch_bounds__(kWarps * 32) append_q8_kernel(const __grid_constant__ AppendQ8Args a) {
    // (cos, sin) of the page's tokens, times the YaRN factor; pair d = 8 part + i at [4 i + part], the rows 4 longer than needed, so
    // that the 16 lanes of a shared-memory access (4 tokens, 4 parts) are on different banks
    __shared__ float2 turn[kPageSize][kHeadDim / 2 + 4];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // a packing that is not 0 <= cu_seqlens[n] <= cu_seqlens[n+1] <= T is reported (one grid-stride pass)
    for (long long n = (long long)blockIdx.x * blockDim.x + threadIdx.x; n < a.N; n += (long long)gridDim.x * blockDim.x) {
        const int c0 = __ldg(&a.cu_seqlens[n]), c1 = __ldg(&a.cu_seqlens[n + 1]);
        if (c0 < 0 || c1 < c0 || c1 > a.T) atomicOr(a.err, kErrBadLength);
    }
    const long long u = blockIdx.x;
    const int n = sequence_of(a.cu_seqlens, a.N, u, lane);
    const int c0 = __ldg(&a.cu_seqlens[n]), c1 = __ldg(&a.cu_seqlens[n + 1]);
    if (c0 < 0 || c1 < c0 || c1 > a.T) return;  // (whole CTA)
    const long long s = __ldg(&a.start_pos[n]), end = s + (c1 - c0);
    const long long pg = (s >> 4) + (u - (((long long)c0 + 30ll * n) >> 4));  // the unit's column of the page table
    const long long p0 = max(s, pg * kPageSize), p1 = min(end, pg * kPageSize + kPageSize);
    if (u < (((long long)c0 + 30ll * n) >> 4) || p0 >= p1) return;
    const int cnt = (int)(p1 - p0), slot0 = (int)(p0 - pg * kPageSize);
    const int t0 = c0 + (int)(p0 - s);  // first token's row
    int page = -1;
    if (pg < 0 || pg >= a.max_pages) {
        if (threadIdx.x == 0) atomicOr(a.err, kErrBadLength);
    } else {
        page = __ldg(&a.page_table[(long long)n * a.max_pages + pg]);
        if (page < 0 || page >= a.num_pages) {
            if (threadIdx.x == 0) atomicOr(a.err, kErrBadPage);
            page = -1;
        }
    }
    if (!kPrologue && page < 0) return;

    // lanes: `wide` tokens of a head at a time (4 lanes each), twice where the page has more than 8
    const int wide = cnt >= 5 ? 8 : cnt >= 3 ? 4 : cnt;
    const int group = 4 * wide, per_warp = 32 / group;
    const int part = lane & 3, tok = (lane >> 2) & (wide - 1), hsub = lane / group, first_lane = lane & ~(group - 1);
    const int heads = kPrologue ? a.Hq + 2 * a.Hkv : 2 * a.Hkv;
    const int rotated = kPrologue ? a.Hq + a.Hkv : 0, Hq = kPrologue ? a.Hq : 0;
    // element offsets of this lane's two 16-byte pieces (as in prologue.cu: its eight pairs are d = 8 part + i)
    const int o0 = kInter ? 16 * part : 8 * part, o1 = kInter ? o0 + 8 : o0 + kHeadDim / 2;

    struct Raw {
        uint4 x[2][2];
    };
    auto load = [&](int hd, Raw& r) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int t = tok + 8 * j;
            if (hd < heads && t < cnt) {
                const __nv_bfloat16* src;
                if (kPrologue) {
                    src = a.qkv + ((long long)(t0 + t) * heads + hd) * kHeadDim;
                } else {
                    src = (hd < a.Hkv ? a.k : a.v) + ((long long)(t0 + t) * a.Hkv + (hd < a.Hkv ? hd : hd - a.Hkv)) * kHeadDim;
                }
                r.x[j][0] = __ldg(reinterpret_cast<const uint4*>(src + o0));
                r.x[j][1] = __ldg(reinterpret_cast<const uint4*>(src + o1));
            } else {
                r.x[j][0] = r.x[j][1] = make_uint4(0, 0, 0, 0);
            }
        }
    };
    const int team = blockIdx.y * kWarps + warp;  // (a unit's heads may be dealt to several CTAs)
    int hd = team * per_warp + hsub;
    const int stride = gridDim.y * kWarps * per_warp;
    Raw cur, nxt;
    load(hd, cur);
    if (kPrologue) {
        for (int i = threadIdx.x; i < cnt * (kHeadDim / 2); i += kWarps * 32) {
            // the angle in double, reduced to [-pi, pi] before a single-precision sincos (as in prologue.cu)
            constexpr double kTwoPi = 6.283185307179586476925286766559, kInvTwoPi = 0.15915494309189533576888376337251;
            double ang = (double)(p0 + i / (kHeadDim / 2)) * a.inv_freq[i % (kHeadDim / 2)];
            ang -= kTwoPi * rint(ang * kInvTwoPi);
            float sn, cs;
            sincosf((float)ang, &sn, &cs);
            const int d = i % (kHeadDim / 2);
            turn[i / (kHeadDim / 2)][4 * (d & 7) + (d >> 3)] = make_float2(cs * a.mscale, sn * a.mscale);
        }
        __syncthreads();
    }

    for (int base = team * per_warp; base < heads; base += stride, hd += stride) {  // (warp-uniform)
        if (base + stride < heads) load(hd + stride, nxt);
        const bool live = hd < heads;
        float u8[2][8], w8[2][8];
        float amax = 0.f;
        bool bad = false;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (j == 1 && cnt <= 8) break;
            const int t = tok + 8 * j;
            float(&x)[8] = u8[j];
            float(&y)[8] = w8[j];
            unpack8(cur.x[j][0], x);
            unpack8(cur.x[j][1], y);
            const bool here = live && t < cnt;
            if (kPrologue && a.bias && here) {
                float bx[8], by[8];
                unpack8(__ldg(reinterpret_cast<const uint4*>(a.bias + hd * kHeadDim + o0)), bx);
                unpack8(__ldg(reinterpret_cast<const uint4*>(a.bias + hd * kHeadDim + o1)), by);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[i] += bx[i];
                    y[i] += by[i];
                }
            }
            if (kPrologue && hd < rotated && here) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 c = turn[t][4 * i + part];
                    // pair i = (x, y): halves (x[i], y[i]); interleaved (x or y)[2(i % 4)], [2(i % 4) + 1]
                    float& p = kInter ? (i < 4 ? x[2 * i] : y[2 * i - 8]) : x[i];
                    float& r = kInter ? (i < 4 ? x[2 * i + 1] : y[2 * i - 7]) : y[i];
                    const float rp = p * c.x - r * c.y, rr = r * c.x + p * c.y;
                    p = rp;
                    r = rr;
                }
            }
            if (here && hd < Hq) {
                uint4* dst = reinterpret_cast<uint4*>(a.q_out + ((long long)(t0 + t) * a.Hq + hd) * kHeadDim);
                dst[o0 / 8] = pack8(x);
                dst[o1 / 8] = pack8(y);
            }
            if (base + per_warp <= Hq) continue;
#pragma unroll
            for (int i = 0; i < 8; ++i) {  // (idle lanes hold zeros)
                const float ax = fabsf(x[i]), ay = fabsf(y[i]);
                bad |= !(ax < kInf) || !(ay < kInf);
                amax = fmaxf(amax, fmaxf(ax < kInf ? ax : 0.f, ay < kInf ? ay : 0.f));
            }
        }
        if (base + per_warp <= Hq || page < 0) {  // query heads only, or no page to write
            cur = nxt;
            continue;
        }
        for (int o = 1; o < group; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const bool writes = live && hd >= Hq;
        const bool is_k = hd < Hq + a.Hkv;
        const int g = hd - Hq - (is_k ? 0 : a.Hkv);
        const long long slice = (long long)page * a.Hkv + g;
        uint8_t* sp = a.kv_scales + slice * 2 + (is_k ? 0 : 1);
        const uint32_t before = writes && slot0 > 0 ? *sp : 0;  // the scale of what the page already holds
        __syncwarp();                                          // (all lanes have it before one replaces it)
        bad |= amax > 448.f * 1099511627776.f;  // (2^40: beyond the largest scale)
        if (writes && bad) atomicOr(a.err, kErrBadValue);
        if (writes) {
            uint8_t* codes = (is_k ? a.k_pages : a.v_pages) + slice * (kPageSize * kHeadDim);
            int e = q8::scale_exp(amax);
            if (slot0 > 0) {  // the page holds tokens of before
                bool off = false;
                const int held = q8::scale_byte(before, off);
                if (off && lane == first_lane) atomicOr(a.err, kErrBadValue);
                if (e > held) {
                    const float f = q8::power(held - e);
                    uint4* row = reinterpret_cast<uint4*>(codes);
                    for (int i = lane - first_lane; i < slot0 * (kHeadDim / 16); i += group) {
                        const uint4 c = row[i];
                        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
                        uint32_t r[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float2 l = q8::floats_of(q8::f16x2_of(w[k])), h = q8::floats_of(q8::f16x2_of_high(w[k]));
                            r[k] = q8::codes_of(l.x * f, l.y * f, h.x * f, h.y * f);
                        }
                        row[i] = make_uint4(r[0], r[1], r[2], r[3]);
                    }
                }
                e = max(e, held);
            }
            const float f = q8::power(-e);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int t = tok + 8 * j;
                if ((j == 1 && cnt <= 8) || t >= cnt) break;
                float(&x)[8] = u8[j];
                float(&y)[8] = w8[j];
                if (bad) {  // an infinity is held as a NaN
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        x[i] += x[i] - x[i];
                        y[i] += y[i] - y[i];
                    }
                }
                uint2* dst = reinterpret_cast<uint2*>(codes + (slot0 + t) * kHeadDim);
                dst[o0 / 8] = make_uint2(q8::codes_of(x[0] * f, x[1] * f, x[2] * f, x[3] * f),
                                         q8::codes_of(x[4] * f, x[5] * f, x[6] * f, x[7] * f));
                dst[o1 / 8] = make_uint2(q8::codes_of(y[0] * f, y[1] * f, y[2] * f, y[3] * f),
                                         q8::codes_of(y[4] * f, y[5] * f, y[6] * f, y[7] * f));
            }
            if (lane == first_lane) *sp = (uint8_t)(e + kScaleBias);
        }
        cur = nxt;
    }
    // this CTA's stores are issued: what is launched behind as a programmatic dependent may start its CTAs
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace

cudaError_t append_q8_launch(const AppendQ8Args& a, cudaStream_t stream) {
    if (a.T == 0 || a.N == 0) return cudaSuccess;
    const long long units = ((long long)a.T + 30ll * a.N) / 16 + 1;
    if (units > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)units, units <= kFewUnits ? 2 : 1);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (!a.qkv) return cudaLaunchKernelEx(&cfg, append_q8_kernel<false, false>, a);
    return a.interleaved ? cudaLaunchKernelEx(&cfg, append_q8_kernel<true, true>, a)
                         : cudaLaunchKernelEx(&cfg, append_q8_kernel<true, false>, a);
}

}  // namespace sinkattn
