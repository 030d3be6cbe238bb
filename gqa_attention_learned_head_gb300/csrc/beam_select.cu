// beam_select.cu -- beam search's selection over beams and vocabulary: log-softmax of every beam's
// logits, the running scores added, the M best continuations of each group.
//
// Mathematics.  score(k, v) = c_k + (z_kv - lse_k), lse_k = ln sum_u e^(z_ku).  Within a row the order of
// the scores is that of the logits, so one pass over a row gives both its sum of exponentials and its M best
// tokens, and only M candidates a row meet the rows of the group.
//   Sum.  Every thread keeps sums of 2^(x L - r) (L = log2 e in 32 bits) against an integer r at or above its
//   largest x L: moving to another r multiplies by a power of two, which is exact, so how a row is cut
//   changes nothing but the order of additions.  Threads hold 32-bit sums of a few hundred terms, everything
//   above that is in 64 bits: the scores of two beams may lie next to each other.  lse = (r + log2 s) / L
//   with the same rounded L, so its rounding cancels to first order.  Where the largest logit is beyond
//   +-2^20 (rows of nothing but a type's lowest value) the share is read again and summed as e^(x - m).
//   Best tokens.  The row is cut into groups of 32 consecutive tokens whose maxima stay in shared memory.  The M
//   best tokens lie in the M best groups (ordered by maximum, then position): of any other group's token there
//   are M tokens ahead.  So the pass over the row has no list to maintain; afterwards the M-th best of the
//   64 maxima that quads of threads have met is a threshold, the groups at or above it (M or a few more) are
//   ranked by counting, and the 32 M tokens of the M best are read again and ranked the same way.  Keys are
//   (order of the value, ~position), all different, so ties need no case of their own.
//
// Two kernels: select_rows_kernel, one CTA per share of a row (rows are cut into as many shares as run at once),
// bound by HBM (one read of the logits) with the exponentials close behind (one MUFU operation per logit);
// select_merge_kernel, one CTA per group, launched as its programmatic dependent.
#include "args_beam.h"
#include "ptx.cuh"

#include <cuda_fp16.h>

namespace sinkattn {
namespace {

constexpr int kThreads = 256;
constexpr int kUnit = 16;             // consecutive tokens that a thread takes at a time: 32 or 64 bytes
constexpr int kGroup = 2 * kUnit;     // tokens of a group, held by two neighbouring threads
constexpr int kQuads = kThreads / 4;  // quads of threads; each quad's best group enters the threshold
static_assert(kQuads >= kBeamMaxSelect, "the threshold needs M maxima");
constexpr float kL = 1.4426950408889634f;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kInf = __builtin_huge_valf();
constexpr float kPlainRange = 1048576.f;  // 2^20: largest |logit| whose x L - r keeps its fraction's worth

// Order of a float as an unsigned number (-0 taken as +0): larger value, larger number; every float's is > 0.
__device__ __forceinline__ unsigned ord32(float x) {
    const unsigned b = __float_as_uint(x + 0.f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float unord32(unsigned o) {
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
// 2^d for an integer-valued d <= 0; 0 below the normal range.
__device__ __forceinline__ float pow2_down(float d) {
    return d < -126.f ? 0.f : __int_as_float((int)(d + 127.f) << 23);
}

template <int DT>
struct Elem;
template <>
struct Elem<kDtF32> {
    using T = float;
    static constexpr unsigned kNone = 0xFF800000u;  // -inf
    __device__ static float get(const T* p) { return __ldcg(p); }
    __device__ static void unpack(const uint32_t (&w)[16], float (&x)[16]) {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(w[i]);
    }
};
template <>
struct Elem<kDtBf16> {
    using T = unsigned short;
    static constexpr unsigned kNone = 0xFF80u;
    __device__ static float get(const T* p) { return __uint_as_float((unsigned)__ldcg(p) << 16); }
    __device__ static void unpack(const uint32_t (&w)[8], float (&x)[16]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
};
template <>
struct Elem<kDtF16> {
    using T = unsigned short;
    static constexpr unsigned kNone = 0xFC00u;
    __device__ static float get(const T* p) { return __half2float(__ushort_as_half(__ldcg(p))); }
    __device__ static void unpack(const uint32_t (&w)[8], float (&x)[16]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
};

// 32 bytes from a 32-byte boundary: one whole sector a thread.
__device__ __forceinline__ void load32(const void* p, uint32_t* r) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "l"(p));
}

// A row's share: where it starts, and which of its units can be read in whole pieces.
template <int DT>
struct Share {
    using E = Elem<DT>;
    using T = typename E::T;
    static constexpr int kWords = kUnit * (int)sizeof(T) / 4;  // 32-bit words of a unit
    const T* p;      // first token of the share
    int len, units;  // tokens, units (the last may be partial)
    int off;         // bytes from the 16-byte boundary at or below p (0..15), the same for every unit
    bool sectors;    // units start at 32-byte boundaries
    int lo, hi;      // units [lo, hi) are whole and their 16-byte pieces lie inside the tensor

    __device__ void set(const T* tensor, const T* tensor_end, const T* first, int n) {
        p = first;
        len = n;
        units = (n + kUnit - 1) / kUnit;
        off = (int)(reinterpret_cast<uintptr_t>(p) & 15);
        sectors = (reinterpret_cast<uintptr_t>(p) & 31) == 0;
        hi = n / kUnit;
        lo = 0;
        if (off) {  // a unit's pieces then start before it and end behind it
            const char* c = reinterpret_cast<const char*>(p) - off;
            if (c < reinterpret_cast<const char*>(tensor)) lo = 1;
            if (hi > 0 && c + hi * (kWords * 4) + 16 > reinterpret_cast<const char*>(tensor_end)) --hi;
        }
    }
    // Unit u's values as words: whole sectors, or 16-byte pieces, shifted together if the row is not aligned to
    // them; token by token at the tensor's edges and past the share's end (-inf there).  The thread that holds a
    // token, and so the order of every sum, does not depend on where the row starts.
    __device__ void load(int u, uint32_t (&w)[kWords]) const {
        if (u >= lo && u < hi) {
            const char* c = reinterpret_cast<const char*>(p) - off + (size_t)u * (kWords * 4);
            const uint4* v = reinterpret_cast<const uint4*>(c);
            if (sectors) {
#pragma unroll
                for (int i = 0; i < kWords / 8; ++i) load32(c + 32 * i, &w[8 * i]);
            } else if (off == 0) {
#pragma unroll
                for (int i = 0; i < kWords / 4; ++i) {
                    const uint4 q = v[i];
                    w[4 * i] = q.x;
                    w[4 * i + 1] = q.y;
                    w[4 * i + 2] = q.z;
                    w[4 * i + 3] = q.w;
                }
            } else {
                uint32_t r[kWords + 4];
#pragma unroll
                for (int i = 0; i < kWords / 4 + 1; ++i) {
                    const uint4 q = v[i];
                    r[4 * i] = q.x;
                    r[4 * i + 1] = q.y;
                    r[4 * i + 2] = q.z;
                    r[4 * i + 3] = q.w;
                }
                if (off & 8) {
#pragma unroll
                    for (int i = 0; i < kWords + 2; ++i) r[i] = r[i + 2];
                }
                if (off & 4) {
#pragma unroll
                    for (int i = 0; i < kWords + 1; ++i) r[i] = r[i + 1];
                }
                if constexpr (sizeof(T) == 4) {
#pragma unroll
                    for (int i = 0; i < kWords; ++i) w[i] = r[i];
                } else {
                    const int bits = 8 * (off & 3);
#pragma unroll
                    for (int i = 0; i < kWords; ++i) w[i] = __funnelshift_r(r[i], r[i + 1], bits);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                if constexpr (sizeof(T) == 4) {
                    const int e = u * kUnit + i;
                    w[i] = e < len ? __float_as_uint(__ldcg(reinterpret_cast<const float*>(p) + e)) : E::kNone;
                } else {
                    const int e = u * kUnit + 2 * i;
                    const unsigned short* h = reinterpret_cast<const unsigned short*>(p);
                    const unsigned a = e < len ? (unsigned)__ldcg(h + e) : E::kNone;
                    const unsigned b = e + 1 < len ? (unsigned)__ldcg(h + e + 1) : E::kNone;
                    w[i] = a | (b << 16);
                }
            }
        }
    }
};

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// How many of the n keys are above `key` (n a multiple of 2, the array 16-byte aligned).
__device__ __forceinline__ int rank_of(const unsigned long long* keys, int n, unsigned long long key) {
    int r = 0;
    const ulonglong2* k2 = reinterpret_cast<const ulonglong2*>(keys);
#pragma unroll 8
    for (int i = 0; i < n / 2; ++i) {
        const ulonglong2 k = k2[i];
        r += (k.x > key) + (k.y > key);
    }
    return r;
}

struct SelectSmem {
    alignas(16) unsigned long long top[kQuads];  // the quads' best groups
    float s[kThreads], r[kThreads];              // the threads' sums and references
    int sel[kBeamMaxSelect];
    unsigned long long threshold;
    int found[2];  // entries of the two lists
};
// Behind it: the groups at or above the threshold (M quads' at most), the tokens of the M best, every group's maximum.
__host__ __device__ inline int groups_of(int tokens) { return (tokens + kGroup - 1) / kGroup; }
__host__ __device__ inline int list_cap(int groups, int M) {  // a quad has two of every 2 kQuads groups
    return M * 2 * ((groups + 2 * kQuads - 1) / (2 * kQuads));
}
__host__ __device__ inline size_t select_smem(int part_len, int M) {
    const int groups = groups_of(part_len);
    return sizeof(SelectSmem) + ((size_t)list_cap(groups, M) + M * kGroup + 2) * 8 + (size_t)groups * 4;
}

template <int DT>
__global__ void __launch_bounds__(kThreads, 4) select_rows_kernel(const BeamArgs a) {
    using E = Elem<DT>;
    using T = typename E::T;
    constexpr int kWords = Share<DT>::kWords;
    constexpr int kBatch = 32 / kWords;  // units loaded together: 128 bytes a thread
    extern __shared__ __align__(16) unsigned char smem_raw[];
    SelectSmem& sm = *reinterpret_cast<SelectSmem*>(smem_raw);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, M = a.M;
    const int row = (int)(blockIdx.x / (unsigned)a.parts), part = (int)(blockIdx.x % (unsigned)a.parts);
    // a finished beam, or one that is not in use, is not read (the merge does not look at its shares)
    if (a.finished && __ldcg(&a.finished[row])) return;
    const float c = __ldcg(&a.scores[row]);
    if (!(c > kNegInf && c < kInf)) return;

    const int e0 = part * a.part_len;
    Share<DT> sh;
    {
        const T* base = static_cast<const T*>(a.logits);
        const T* end = base + ((long long)a.N * a.K - 1) * a.row_stride + a.V;
        sh.set(base, end, base + row * a.row_stride + e0, min(a.part_len, a.V - e0));
    }
    const int groups = groups_of(sh.len);
    unsigned long long* list = reinterpret_cast<unsigned long long*>(&sm + 1);
    unsigned long long* tokens = list + list_cap(groups_of(a.part_len), M);
    float* gmax = reinterpret_cast<float*>(tokens + M * kGroup + 2);

    // ---- 1. one pass over the share: sums, and every group's maximum.  A group is two neighbouring threads' units.
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    float r2 = -1e9f, best = kNegInf;
    int best_g = 0;
    for (int u0 = tid; u0 - lane < sh.units; u0 += kThreads * kBatch) {  // whole warps
        uint32_t w[kBatch][kWords];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int u = u0 + b * kThreads;
            if (u < sh.units) {
                sh.load(u, w[b]);
            } else {
#pragma unroll
                for (int i = 0; i < kWords; ++i) w[b][i] = sizeof(T) == 4 ? E::kNone : E::kNone * 0x10001u;
            }
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int u = u0 + b * kThreads;
            float x[kUnit];
            E::unpack(w[b], x);
            float m4[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) m4[i] = fmaxf(fmax3(x[4 * i], x[4 * i + 1], x[4 * i + 2]), x[4 * i + 3]);
            float gm = fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]);
            gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, 1));  // the other half of the group
            if (!(tid & 1) && u < sh.units) gmax[u >> 1] = gm;
            if (gm > best) {
                best = gm;
                best_g = u >> 1;
                const float r = ceilf(gm * kL);
                if (r > r2) {
                    const float f = pow2_down(r2 - r);
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[i] *= f;
                    r2 = r;
                }
            }
#pragma unroll
            for (int i = 0; i < kUnit; ++i) s[i & 3] += fast_exp2(fmaf(x[i], kL, -r2));
        }
    }
    sm.s[tid] = (s[0] + s[1]) + (s[2] + s[3]);
    sm.r[tid] = r2;
    unsigned long long top = best > kNegInf ? ((unsigned long long)ord32(best) << 32) | (unsigned)~best_g : 0ull;
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        const unsigned long long y = __shfl_xor_sync(0xffffffffu, top, o);
        top = y > top ? y : top;
    }
    const bool none = top == 0;
    if (none) top = (unsigned long long)(kQuads - 1 - (tid >> 2));  // below every group, and different in every quad
    if ((lane & 3) == 0) sm.top[tid >> 2] = top;
    if (tid < 2) sm.found[tid] = 0;
    __syncthreads();

    // ---- 2. the share's maximum; its sum again against that maximum where it is far out
    float m_all;
    {
        const unsigned long long x = sm.top[lane], y = sm.top[lane + 32];
        const unsigned o = __reduce_max_sync(0xffffffffu, (unsigned)((x > y ? x : y) >> 32));
        m_all = o ? unord32(o) : kNegInf;
    }
    const bool far = m_all > kPlainRange || (m_all < -kPlainRange && m_all != kNegInf);
    if (far) {
        float t = 0.f;
        for (int u = tid; u < sh.units; u += kThreads) {
            uint32_t w[kWords];
            float x[kUnit];
            sh.load(u, w);
            E::unpack(w, x);
#pragma unroll
            for (int i = 0; i < kUnit; ++i) t += fast_exp2((x[i] - m_all) * kL);
        }
        sm.s[tid] = t;
        __syncthreads();
    }

    // ---- 3. the threshold: the M-th best of the quads' best groups; meanwhile the last warp adds the sums up
    if (tid < kQuads) {
        const unsigned long long key = sm.top[tid];
        if (rank_of(sm.top, kQuads, key) == M - 1) sm.threshold = key;
    } else if (warp == kThreads / 32 - 1) {
        float r = kNegInf;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) r = fmaxf(r, sm.r[lane + 32 * i]);
        r = warp_max(r);
        double t = 0.0;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i)  // scaled by exact powers of two (a NaN stays one)
            t += (double)(far ? sm.s[lane + 32 * i] : sm.s[lane + 32 * i] * pow2_down(sm.r[lane + 32 * i] - r));
        t = warp_sum(t);
        if (lane == 0) {
            BeamPart out;
            out.r2 = far ? kInf : r;
            out.m = m_all;
            out.s = t;
            a.part[blockIdx.x] = out;
        }
    }
    __syncthreads();
    const unsigned long long thr = sm.threshold;
    if (!none && top >= thr && !(lane & 1)) {
        for (int g = tid >> 1; g < groups; g += kThreads / 2) {
            const float v = gmax[g];
            const unsigned long long key = ((unsigned long long)ord32(v) << 32) | (unsigned)~g;
            if (key >= thr && v > kNegInf) list[atomicAdd(&sm.found[0], 1)] = key;
        }
    }
    __syncthreads();
    const int n = sm.found[0];  // <= M x (groups of a quad)
    for (int i = tid; i < n; i += kThreads) {
        const unsigned long long key = list[i];
        int r = rank_of(list, n & ~1, key);
        if (n & 1) r += list[n - 1] > key;
        if (r < M) sm.sel[r] = (int)~(unsigned)key;
    }
    __syncthreads();

    // ---- 4. the tokens of the best groups that can be among the M best, ranked
    const unsigned thr_v = (unsigned)(thr >> 32);
    for (int i = tid; i < min(n, M) * kGroup; i += kThreads) {
        const int e = sm.sel[i / kGroup] * kGroup + i % kGroup;
        if (e >= sh.len) continue;
        const float v = E::get(sh.p + e);
        const unsigned o = ord32(v);
        if (v > kNegInf && o >= thr_v)
            tokens[atomicAdd(&sm.found[1], 1)] = ((unsigned long long)o << 32) | (unsigned)~(e0 + e);
    }
    __syncthreads();
    const int nt = sm.found[1];
    unsigned long long* out = a.best + (size_t)blockIdx.x * M;
    for (int i = tid; i < nt; i += kThreads) {
        const unsigned long long key = tokens[i];
        int r = rank_of(tokens, nt & ~1, key);
        if (nt & 1) r += tokens[nt - 1] > key;
        if (r < M) out[r] = key;
    }
    if (tid >= nt && tid < M) out[tid] = 0;
}

// ---------------------------------------------------------------------------- merge over a group's rows
// Order of a continuation: its score's order, then ~(beam, token).
struct Cand {
    unsigned long long score, at;
    __device__ bool above(const Cand& o) const { return score > o.score || (score == o.score && at > o.at); }
};
__device__ __forceinline__ unsigned long long ord64(double x) {
    const unsigned long long b = (unsigned long long)__double_as_longlong(x + 0.0);
    return (b >> 63) ? ~b : (b | (1ull << 63));
}
__device__ __forceinline__ double unord64(unsigned long long o) {
    return __longlong_as_double((long long)((o >> 63) ? (o & ~(1ull << 63)) : ~o));
}

// log2 of a positive normal number, to about 2^-44: 2^e m with m in [sqrt(1/2), sqrt(2)), and the series of
// ln m = 2 artanh t, t = (m - 1) / (m + 1), |t| < 0.172, cut behind t^13 / 13 (the next term is below 3e-13).  Sixteen
// 64-bit operations: they are slow on this GPU.
__device__ __forceinline__ double log2_series(double s) {
    const long long b = __double_as_longlong(s);
    int e = (int)((b >> 52) & 0x7ff) - 1023;
    double m = __longlong_as_double((b & 0x000fffffffffffffll) | 0x3ff0000000000000ll);
    if (m > 1.4142135623730951) {
        m *= 0.5;
        ++e;
    }
    const double den = m + 1.0;
    double inv = (double)__frcp_rn((float)den);
    inv = inv * (2.0 - den * inv);  // one Newton step: 2^-24 squared
    const double t = (m - 1.0) * inv, q = t * t;
    double p = 1.0 / 13.0;
    p = p * q + 1.0 / 11.0;
    p = p * q + 1.0 / 9.0;
    p = p * q + 1.0 / 7.0;
    p = p * q + 1.0 / 5.0;
    p = p * q + 1.0 / 3.0;
    p = p * q + 1.0;
    return (double)e + 2.8853900817779268 * (t * p);  // 2 / ln 2
}

struct MergeSmem {
    alignas(16) Cand top[kQuads];
    double lse[kBeamMaxBeams];
    float cum[kBeamMaxBeams];
    int state[kBeamMaxBeams];  // 0: no continuation, 1: read, 2: finished
    Cand threshold;
    int found;
};
// Behind it: the K x parts x M candidates, and the numbers of those at or above the threshold.
inline size_t merge_smem(int total) { return sizeof(MergeSmem) + (size_t)total * (sizeof(Cand) + 4); }

__global__ void __launch_bounds__(kThreads) select_merge_kernel(const BeamArgs a) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    MergeSmem& sm = *reinterpret_cast<MergeSmem*>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = blockIdx.x;
    const int K = a.K, M = a.M, parts = a.parts, total = K * parts * M;
    Cand* cands = reinterpret_cast<Cand*>(&sm + 1);
    int* list = reinterpret_cast<int*>(cands + total);
    if (tid == 0) sm.found = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- 1. each row's log-sum-exp from its shares: a warp per row, a lane per share
    for (int k = warp; k < K; k += kThreads / 32) {
        const long long row = (long long)n * K + k;
        const float c = __ldcg(&a.scores[row]);
        const bool done = a.finished && __ldcg(&a.finished[row]);
        int st = c > kNegInf && c < kInf ? (done ? 2 : 1) : 0;
        bool bad = c != c || c == kInf;
        double l = 0.0;
        if (st == 1) {
            const BeamPart* p = a.part + row * parts;
            float m = kNegInf, r = -1e9f;
            bool far = false, nan = false;
            for (int i = lane; i < parts; i += 32) {
                const float ri = __ldcg(&p[i].r2);
                const double si = __ldcg(&p[i].s);
                m = fmaxf(m, __ldcg(&p[i].m));
                far = far || ri == kInf;
                r = ri == kInf ? r : fmaxf(r, ri);
                nan = nan || si != si;
            }
            m = warp_max(m);
            r = warp_max(r);
            far = __any_sync(0xffffffffu, far);
            nan = __any_sync(0xffffffffu, nan);
            if (nan || m == kInf) {
                bad = true;
                st = 0;
            } else if (m == kNegInf) {  // every token is masked
                st = 0;
            } else if (!far) {
                double sum = 0.0;
                for (int i = lane; i < parts; i += 32) sum += __ldcg(&p[i].s) * (double)pow2_down(__ldcg(&p[i].r2) - r);
                l = ((double)r + log2_series(warp_sum(sum))) * (1.0 / (double)kL);
            } else {
                double sum = 0.0;
                for (int i = lane; i < parts; i += 32) {
                    const float mi = __ldcg(&p[i].m), ri = __ldcg(&p[i].r2);
                    if (mi == kNegInf) continue;
                    const double li = ri == kInf ? (double)mi + log(__ldcg(&p[i].s))
                                                 : ((double)ri + log2_series(__ldcg(&p[i].s))) * (1.0 / (double)kL);
                    sum += exp(li - (double)m);
                }
                l = (double)m + log(warp_sum(sum));
            }
        }
        if (lane == 0) {
            if (bad) atomicOr(a.err, kErrBadValue);
            sm.lse[k] = l;
            sm.cum[k] = c;
            sm.state[k] = st;
        }
    }
    __syncthreads();

    // ---- 2. the candidates; the M-th best of the quads' best bounds the M-th best of all
    Cand mine = {0ull, 0ull};
    for (int i = tid; i < total; i += kThreads) {
        Cand x = {0ull, 0ull};
        const int k = i / (parts * M), st = sm.state[k];
        if (st == 1) {
            const unsigned long long key = __ldcg(&a.best[(long long)n * total + i]);
            if (key) {
                const double z = unord32((unsigned)(key >> 32));
                x.score = ord64((double)sm.cum[k] + (z - sm.lse[k]));
                x.at = ~(((unsigned long long)k << 32) | ~(unsigned)key);
            }
        } else if (st == 2 && i == k * parts * M) {
            x.score = ord64((double)sm.cum[k]);
            x.at = ~(((unsigned long long)k << 32) | (unsigned)a.pad_token);
        }
        cands[i] = x;
        if (x.above(mine)) mine = x;
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        Cand y;
        y.score = __shfl_xor_sync(0xffffffffu, mine.score, o);
        y.at = __shfl_xor_sync(0xffffffffu, mine.at, o);
        if (y.above(mine)) mine = y;
    }
    if (!mine.score) mine.at = (unsigned long long)(kQuads - 1 - (tid >> 2));  // none, but different in every quad
    if ((lane & 3) == 0) sm.top[tid >> 2] = mine;
    __syncthreads();
    if (tid < kQuads) {
        const Cand x = sm.top[tid];
        int r = 0;
#pragma unroll 8
        for (int i = 0; i < kQuads; ++i) r += sm.top[i].above(x);
        if (r == M - 1) sm.threshold = x;
    }
    __syncthreads();
    const Cand thr = sm.threshold;
    if (mine.score && !thr.above(mine)) {
        for (int i = tid; i < total; i += kThreads) {
            const Cand x = cands[i];
            if (x.score && !thr.above(x)) list[atomicAdd(&sm.found, 1)] = i;
        }
    }
    __syncthreads();

    // ---- 3. ranked by counting
    const int found = sm.found;
    for (int i = tid; i < found; i += kThreads) {
        const Cand x = cands[list[i]];
        int q = 0;
#pragma unroll 4
        for (int j = 0; j < found; ++j) q += cands[list[j]].above(x);
        if (q < M) {
            const unsigned long long at = ~x.at;
            a.out_scores[(long long)n * M + q] = (float)unord64(x.score);
            a.out_parents[(long long)n * M + q] = n * K + (int)(at >> 32);
            a.out_tokens[(long long)n * M + q] = (int)(unsigned)at;
        }
    }
    if (tid >= found && tid < M) {
        a.out_scores[(long long)n * M + tid] = kNegInf;
        a.out_parents[(long long)n * M + tid] = -1;
        a.out_tokens[(long long)n * M + tid] = -1;
    }
}

// Shared memory that a kernel may be launched with, raised once per device and thread as calls ask for more.
cudaError_t allow_smem(const void* kernel, int which, size_t bytes) {
    static thread_local size_t allowed[64][4] = {};
    if (bytes <= 48 * 1024) return cudaSuccess;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && allowed[dev][which] >= bytes) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess && dev < 64) allowed[dev][which] = bytes;
    return e;
}

}  // namespace

cudaError_t beam_plan(int N, int K, int V, int M, BeamPlan* plan) {
    int sms = 0, dev = 0;
    cudaError_t e;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    const long long rows = (long long)N * K;
    // shares of a row: as many as run at once (four CTAs an SM), but none below 4096 tokens (one step of a thread)
    long long parts = rows > 0 ? (4ll * sms) / rows : 1;
    const long long fine = V / 4096;
    if (parts > fine) parts = fine;
    const long long least = (V + kBeamMaxPart - 1) / kBeamMaxPart;
    if (parts > kBeamMaxCands / 2 / ((long long)K * M)) parts = kBeamMaxCands / 2 / ((long long)K * M);
    if (parts < least) parts = least;
    if (parts < 1) parts = 1;
    const long long len = ((V + parts - 1) / parts + kGroup - 1) / kGroup * kGroup;
    plan->part_len = (int)len;
    plan->parts = (int)((V + len - 1) / len);
    size_t bytes = (size_t)rows * plan->parts * sizeof(BeamPart);
    plan->best_offset = (bytes + 255) & ~size_t(255);
    plan->ws_bytes = plan->best_offset + (size_t)rows * plan->parts * M * sizeof(unsigned long long);
    return cudaSuccess;
}

cudaError_t beam_select_launch(const BeamArgs& a, cudaStream_t stream) {
    const long long units = (long long)a.N * a.K * a.parts;
    if (units == 0) return cudaSuccess;
    if (units > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)units);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = select_smem(a.part_len, a.M);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void (*rows)(const BeamArgs) = a.dtype == kDtF32    ? select_rows_kernel<kDtF32>
                                   : a.dtype == kDtBf16 ? select_rows_kernel<kDtBf16>
                                                        : select_rows_kernel<kDtF16>;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(rows), a.dtype, cfg.dynamicSmemBytes);
    if (e != cudaSuccess) return e;
    if ((e = cudaLaunchKernelEx(&cfg, rows, a)) != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)a.N);
    cfg.dynamicSmemBytes = merge_smem(a.K * a.parts * a.M);
    if ((e = allow_smem(reinterpret_cast<const void*>(select_merge_kernel), 3, cfg.dynamicSmemBytes)) != cudaSuccess)
        return e;
    return cudaLaunchKernelEx(&cfg, select_merge_kernel, a);
}

}  // namespace sinkattn
