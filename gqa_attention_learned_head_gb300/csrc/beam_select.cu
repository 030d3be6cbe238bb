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
//   Best tokens.  The row is cut into groups of 16 tokens whose maxima stay in shared memory.  The M best
//   tokens lie in the M best groups (ordered by maximum, then position): of any other group's token there
//   are M tokens ahead.  So the pass over the row has no list to maintain; afterwards the M best of the
//   threads' maxima give a threshold, the groups at or above it (M or a few more) are ranked by counting,
//   and the 16 M tokens of the M best are read again and ranked the same way.  Keys are (order of the value,
//   ~position), all different, so ties need no case of their own.
//
// Two kernels: select_rows_kernel, one CTA per share of a row (a row is cut into as many shares as fill the
// GPU), bound by HBM (one read of the logits) with the exponentials close behind (one MUFU operation per
// logit); select_merge_kernel, one CTA per group, launched as its programmatic dependent.
#include "args_beam.h"
#include "ptx.cuh"

#include <cuda_fp16.h>

namespace sinkattn {
namespace {

constexpr int kThreads = 256;
constexpr int kGroup = 16;  // tokens of a group: 32 or 64 bytes, a thread's loads of one step
constexpr int kMaxGroups = kBeamMaxPart / kGroup;
constexpr int kListCap = kBeamMaxSelect * kMaxGroups / kThreads;  // at most M threads' groups pass the threshold
static_assert(kListCap >= kBeamMaxSelect * kGroup, "the token list uses the group list's room");
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

// A row's share: where it starts, and which of its groups can be read in 16-byte pieces.
template <int DT>
struct Share {
    using E = Elem<DT>;
    using T = typename E::T;
    static constexpr int kWords = kGroup * (int)sizeof(T) / 4;  // 32-bit words of a group
    const T* p;       // first token of the share
    int len, groups;  // tokens, groups (the last may be partial)
    int off;          // bytes from the 16-byte boundary at or below p (0..15), the same for every group
    int lo, hi;       // groups [lo, hi) are whole and their 16-byte pieces lie inside the tensor

    __device__ void set(const T* tensor, const T* tensor_end, const T* first, int n) {
        p = first;
        len = n;
        groups = (n + kGroup - 1) / kGroup;
        off = (int)(reinterpret_cast<uintptr_t>(p) & 15);
        hi = n / kGroup;
        lo = 0;
        if (off) {  // a group's pieces then start before it and end behind it
            const char* c = reinterpret_cast<const char*>(p) - off;
            if (c < reinterpret_cast<const char*>(tensor)) lo = 1;
            if (hi > 0 && c + hi * (kWords * 4) + 16 > reinterpret_cast<const char*>(tensor_end)) --hi;
        }
    }
    // Group g's values as words: 16-byte pieces, shifted together if the row is not aligned to them; token by
    // token at the tensor's edges and past the share's end (-inf there).
    __device__ void load(int g, uint32_t (&w)[kWords]) const {
        if (g >= lo && g < hi) {
            const uint4* v = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(p) - off + (size_t)g * (kWords * 4));
            if (off == 0) {
#pragma unroll
                for (int i = 0; i < kWords / 4; ++i) {
                    const uint4 q = __ldcg(v + i);
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
                const int bits = 8 * (off & 3);
#pragma unroll
                for (int i = 0; i < kWords; ++i) w[i] = __funnelshift_r(r[i], r[i + 1], bits);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                if constexpr (sizeof(T) == 4) {
                    const int e = g * kGroup + i;
                    w[i] = e < len ? __float_as_uint(__ldcg(reinterpret_cast<const float*>(p) + e)) : E::kNone;
                } else {
                    const int e = g * kGroup + 2 * i;
                    const unsigned a = e < len ? (unsigned)__ldcg(reinterpret_cast<const unsigned short*>(p) + e) : E::kNone;
                    const unsigned b =
                        e + 1 < len ? (unsigned)__ldcg(reinterpret_cast<const unsigned short*>(p) + e + 1) : E::kNone;
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
#pragma unroll 4
    for (int i = 0; i < n / 2; ++i) {
        const ulonglong2 k = k2[i];
        r += (k.x > key) + (k.y > key);
    }
    return r;
}

struct SelectSmem {
    alignas(16) unsigned long long top[kThreads];  // the threads' best groups
    alignas(16) unsigned long long list[kListCap + 2];
    float gmax[kMaxGroups];
    int sel[kBeamMaxSelect];
    unsigned long long threshold;
    float red_m[kThreads / 32], red_r[kThreads / 32];
    double red_s[kThreads / 32];
    int count;
};

template <int DT>
__global__ void __launch_bounds__(kThreads) select_rows_kernel(const BeamArgs a) {
    using E = Elem<DT>;
    using T = typename E::T;
    constexpr int kWords = Share<DT>::kWords;
    constexpr int kBatch = 32 / kWords;  // groups loaded together: 128 bytes a thread
    __shared__ SelectSmem sm;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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

    // ---- 1. one pass over the share: sums, and every group's maximum
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    float r2 = -1e9f, best = kNegInf;
    int best_g = 0;
    for (int g0 = tid; g0 < sh.groups; g0 += kThreads * kBatch) {
        uint32_t w[kBatch][kWords];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int g = g0 + u * kThreads;
            if (g < sh.groups) {
                sh.load(g, w[u]);
            } else {
#pragma unroll
                for (int i = 0; i < kWords; ++i) w[u][i] = sizeof(T) == 4 ? E::kNone : E::kNone * 0x10001u;
            }
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int g = g0 + u * kThreads;
            float x[kGroup];
            E::unpack(w[u], x);
            float m4[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) m4[i] = fmaxf(fmax3(x[4 * i], x[4 * i + 1], x[4 * i + 2]), x[4 * i + 3]);
            const float gm = fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]);
            if (g < sh.groups) sm.gmax[g] = gm;
            if (gm > best) {
                best = gm;
                best_g = g;
                const float r = ceilf(gm * kL);
                if (r > r2) {
                    const float f = pow2_down(r2 - r);
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[i] *= f;
                    r2 = r;
                }
            }
#pragma unroll
            for (int i = 0; i < kGroup; ++i) s[i & 3] += fast_exp2(fmaf(x[i], kL, -r2));
        }
    }

    // ---- 2. the share's maximum and sum
    float m_all, r_all;
    {
        const float wm = warp_max(best), wr = warp_max(r2);
        if (lane == 0) {
            sm.red_m[warp] = wm;
            sm.red_r[warp] = wr;
        }
        sm.top[tid] = best > kNegInf ? ((unsigned long long)ord32(best) << 32) | (unsigned)~best_g
                                     : (unsigned long long)(kThreads - 1 - tid);
        if (tid == 0) sm.count = 0;
        __syncthreads();
        m_all = sm.red_m[0];
        r_all = sm.red_r[0];
#pragma unroll
        for (int i = 1; i < kThreads / 32; ++i) {
            m_all = fmaxf(m_all, sm.red_m[i]);
            r_all = fmaxf(r_all, sm.red_r[i]);
        }
    }
    float mine = (s[0] + s[1]) + (s[2] + s[3]);
    const bool far = m_all > kPlainRange || (m_all < -kPlainRange && m_all != kNegInf);
    if (far) {
        mine = 0.f;
        for (int g = tid; g < sh.groups; g += kThreads) {
            uint32_t w[kWords];
            float x[kGroup];
            sh.load(g, w);
            E::unpack(w, x);
#pragma unroll
            for (int i = 0; i < kGroup; ++i) mine += fast_exp2((x[i] - m_all) * kL);
        }
    } else {
        mine *= pow2_down(r2 - r_all);  // keeps a NaN
    }
    {
        const double ws = warp_sum((double)mine);
        if (lane == 0) sm.red_s[warp] = ws;
    }

    // ---- 3. the groups at or above the M-th best of the threads' best groups
    const int M = a.M;
    const unsigned long long my_top = sm.top[tid];
    if (rank_of(sm.top, kThreads, my_top) == M - 1) sm.threshold = my_top;
    __syncthreads();
    if (tid == 0) {
        double t = sm.red_s[0];
#pragma unroll
        for (int i = 1; i < kThreads / 32; ++i) t += sm.red_s[i];
        BeamPart out;
        out.r2 = far ? kInf : r_all;
        out.m = m_all;
        out.s = t;
        a.part[blockIdx.x] = out;
    }
    const unsigned long long thr = sm.threshold;
    if (my_top >= thr && best > kNegInf) {
        for (int g = tid; g < sh.groups; g += kThreads) {
            const float v = sm.gmax[g];
            const unsigned long long key = ((unsigned long long)ord32(v) << 32) | (unsigned)~g;
            if (key >= thr && v > kNegInf) sm.list[atomicAdd(&sm.count, 1)] = key;
        }
    }
    __syncthreads();
    int n = sm.count;  // <= M x (groups per thread) <= kListCap
    if (tid == 0) sm.list[n] = 0;  // an even count for the ranking
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
        const unsigned long long key = sm.list[i];
        const int r = rank_of(sm.list, (n + 1) & ~1, key);
        if (r < M) sm.sel[r] = (int)~(unsigned)key;
    }
    const int n_sel = min(n, M);
    __syncthreads();  // the list and its count are free again
    if (tid == 0) sm.count = 0;
    __syncthreads();

    // ---- 4. the tokens of those groups that can be among the M best, ranked
    const unsigned thr_v = (unsigned)(thr >> 32);
    for (int i = tid; i < n_sel * kGroup; i += kThreads) {
        const int e = sm.sel[i / kGroup] * kGroup + i % kGroup;
        if (e >= sh.len) continue;
        const float v = E::get(sh.p + e);
        const unsigned o = ord32(v);
        if (v > kNegInf && o >= thr_v)
            sm.list[atomicAdd(&sm.count, 1)] = ((unsigned long long)o << 32) | (unsigned)~(e0 + e);
    }
    __syncthreads();
    n = sm.count;
    if (tid == 0) sm.list[n] = 0;
    __syncthreads();
    unsigned long long* out = a.best + (size_t)blockIdx.x * M;
    for (int i = tid; i < n; i += kThreads) {
        const unsigned long long key = sm.list[i];
        const int r = rank_of(sm.list, (n + 1) & ~1, key);
        if (r < M) out[r] = key;
    }
    if (tid >= n && tid < M) out[tid] = 0;
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

// at most M threads pass the threshold, each with its share of the K x parts x M candidates
constexpr int kMergeCap = kBeamMaxSelect * kBeamMaxCands / kThreads;

__global__ void __launch_bounds__(kThreads) select_merge_kernel(const BeamArgs a) {
    __shared__ double lse[kBeamMaxBeams];
    __shared__ float cum[kBeamMaxBeams];
    __shared__ int state[kBeamMaxBeams];  // 0: no continuation, 1: read, 2: finished
    __shared__ Cand top[kThreads];
    __shared__ Cand list[kMergeCap];
    __shared__ Cand threshold;
    __shared__ int count;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, n = blockIdx.x;
    const int K = a.K, M = a.M, parts = a.parts, total = K * parts * M;

    // ---- 1. each row's log-sum-exp from its shares
    if (tid == 0) count = 0;
    if (tid < K) {
        const long long row = (long long)n * K + tid;
        const float c = __ldcg(&a.scores[row]);
        int st = c > kNegInf && c < kInf ? 1 : 0;
        if (c != c || c == kInf) atomicOr(a.err, kErrBadValue);
        if (st && a.finished && __ldcg(&a.finished[row])) st = 2;
        double l = 0.0;
        if (st == 1) {
            const BeamPart* p = a.part + row * parts;
            float m = kNegInf, r = -1e9f;
            bool far = false, nan = false;
            for (int i = 0; i < parts; ++i) {
                m = fmaxf(m, __ldcg(&p[i].m));
                const float ri = __ldcg(&p[i].r2);
                if (ri == kInf) far = true;
                else r = fmaxf(r, ri);
                nan = nan || __ldcg(&p[i].s) != __ldcg(&p[i].s);
            }
            if (nan || m == kInf) {
                atomicOr(a.err, kErrBadValue);
                st = 0;
            } else if (m == kNegInf) {  // every token is masked
                st = 0;
            } else if (!far) {
                double sum = 0.0;
                for (int i = 0; i < parts; ++i) sum += __ldcg(&p[i].s) * (double)pow2_down(__ldcg(&p[i].r2) - r);
                l = ((double)r + log2(sum)) / (double)kL;
            } else {
                double sum = 0.0;
                for (int i = 0; i < parts; ++i) {
                    const float mi = __ldcg(&p[i].m), ri = __ldcg(&p[i].r2);
                    if (mi == kNegInf) continue;
                    const double li = ri == kInf ? (double)mi + log(__ldcg(&p[i].s))
                                                 : ((double)ri + log2(__ldcg(&p[i].s))) / (double)kL;
                    sum += exp(li - (double)m);
                }
                l = (double)m + log(sum);
            }
        }
        lse[tid] = l;
        cum[tid] = c;
        state[tid] = st;
    }
    __syncthreads();

    // ---- 2. every thread's best continuation; the M-th best of them bounds the M-th best of all
    auto cand = [&](int i) {
        Cand r = {0ull, 0ull};
        const int k = i / (parts * M), st = state[k];
        if (st == 1) {
            const unsigned long long key = __ldcg(&a.best[((long long)n * K * parts) * M + i]);
            if (key) {
                const double z = unord32((unsigned)(key >> 32));
                r.score = ord64((double)cum[k] + (z - lse[k]));
                r.at = ~(((unsigned long long)k << 32) | ~(unsigned)key);
            }
        } else if (st == 2 && i == k * parts * M) {
            r.score = ord64((double)cum[k]);
            r.at = ~(((unsigned long long)k << 32) | (unsigned)a.pad_token);
        }
        return r;
    };
    Cand mine = {0ull, (unsigned long long)(kThreads - 1 - tid)};  // none, but different in every thread
    for (int i = tid; i < total; i += kThreads) {
        const Cand x = cand(i);
        if (x.score && x.above(mine)) mine = x;
    }
    top[tid] = mine;
    __syncthreads();
    int r = 0;
    for (int i = 0; i < kThreads; ++i) r += top[i].above(mine);
    if (r == M - 1) threshold = mine;
    __syncthreads();
    const Cand thr = threshold;
    if (!thr.above(mine) && mine.score) {
        for (int i = tid; i < total; i += kThreads) {
            const Cand x = cand(i);
            if (x.score && !thr.above(x)) list[atomicAdd(&count, 1)] = x;
        }
    }
    __syncthreads();
    const int found = count;
    for (int i = tid; i < found; i += kThreads) {
        const Cand x = list[i];
        int q = 0;
        for (int j = 0; j < found; ++j) q += list[j].above(x);
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

}  // namespace

cudaError_t beam_plan(int N, int K, int V, int M, BeamPlan* plan) {
    int sms = 0, dev = 0;
    cudaError_t e;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    const long long rows = (long long)N * K;
    // shares of a row: enough to give every SM four CTAs, but not below 4096 tokens (a thread's one step)
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
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = a.dtype == kDtF32    ? cudaLaunchKernelEx(&cfg, select_rows_kernel<kDtF32>, a)
                    : a.dtype == kDtBf16 ? cudaLaunchKernelEx(&cfg, select_rows_kernel<kDtBf16>, a)
                                                  : cudaLaunchKernelEx(&cfg, select_rows_kernel<kDtF16>, a);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)a.N);
    return cudaLaunchKernelEx(&cfg, select_merge_kernel, a);
}

}  // namespace sinkattn
