// beam_select.cu -- beam search's selection over beams and vocabulary: log-softmax of every beam's
// logits, the running scores added, the M best continuations of each group.
//
// Mathematics.  score(k, v) = c_k + (z_kv - lse_k), lse_k = ln sum_u e^(z_ku).  Within a row the order of
// the scores is that of the logits, so one pass over a row gives both its sum of exponentials and its M best
// tokens, and only M candidates a row meet the rows of the group.
//   Sum.  Every thread keeps sums of 2^(x L - r) (L = log2 e in 32 bits) against an integer r near its
//   largest x L: moving to another r multiplies by a power of two, which is exact, so how a row is cut
//   changes nothing but the order of additions.  Threads hold 32-bit sums of up to 1024 terms, everything above that is in
//   pairs of floats (48 bits) and adds nothing to their error.  lse = (r + log2 s) / L with the same rounded L: what its
//   rounding does to the exponents cancels but for 1.3e-8 of the row's entropy.  So the logarithm of the sum is off by at
//   most 8e-6 (four sums of 256 additions a thread in a share of 262144 tokens, were all roundings to lean one way; 5e-6 up to
//   131072; on random rows none of it shows beside the rounding of a 32-bit score), and beams whose scores are closer than
//   twice that may come in either order.  Where the largest logit is beyond +-2^20 (rows of nothing but a type's lowest value) the share
//   is read again and summed as e^(x - m), one sum a thread: 3.1e-5.
//   Best tokens.  The row is cut into groups of 32 consecutive tokens whose maxima stay in shared memory.  The M
//   best tokens lie in the M best groups (ordered by maximum, then position): of any other group's token there
//   are M tokens ahead.  So the pass over the row has no list to maintain; afterwards the M-th best of the
//   maxima that teams of threads have met is a threshold, the groups at or above it (M or a few more) are
//   ranked by counting, and the 32 M tokens of the M best are read again and ranked the same way.  Keys are
//   (order of the value, ~position), all different, so ties need no case of their own.
//
// Two kernels: select_rows_kernel, one CTA per share of a row (rows are cut into as many shares as run at once),
// bound by HBM (one read of the logits) with the exponentials close behind (one MUFU operation per logit);
// select_merge_kernel, one CTA per group, launched as its programmatic dependent.
//
// Measured (GB300, calls back to back from a graph): 64 groups of 8 rows of 200000 bf16 logits 43 us, 4.8 TB/s = 70% of
// the copy rate: the pass over the rows takes 29 us (7 TB/s), its tail (threshold, 64 x 32 tokens read again and ranked)
// 5 us, the merge 3.5, the rest is starts; f16 the same.  32 groups of 8 rows of 50021 f32 logits 18.7 us (51 MB: 7.5 us of
// reading), f16 14.9; one group of 4 rows of 32000 7.9 us in any type, all latency.  Five or six CTAs an SM (fewer registers,
// spills) and more, smaller shares were slower; 64-bit sums and 128-bit keys in the merge took 19.5 us where pairs of floats take 3.5.
#include "args_beam.h"
#include "errors_beam.h"
#include "ptx.cuh"

#include <cuda_fp16.h>

namespace sinkattn {
namespace {

constexpr int kThreads = 256;
constexpr int kUnit = 16;             // consecutive tokens that a thread takes at a time: 32 or 64 bytes
constexpr int kGroup = 2 * kUnit;     // tokens of a group, held by two neighbouring threads
// The M-th best of what teams of threads have met is a threshold: 64 teams of four for up to 32 picks, else 128 of two (as
// many teams as picks would leave several hundred above it).
constexpr int kMaxTeams = kThreads / 2;
static_assert(kThreads / 4 >= 2 * 32 && kMaxTeams >= 2 * kBeamMaxSelect, "twice as many teams as picks");
__device__ __forceinline__ int team_of(int M) { return M > 32 ? 2 : 4; }
constexpr float kL = 1.4426950408889634f;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kInf = __builtin_huge_valf();
constexpr float kSlack = 16.f;  // log2 units that a thread's largest exponential may be above its reference
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
    __device__ static T put(float x) { return x; }  // a value of the type as T, exact
    __device__ static float at(T x) { return x; }
    __device__ static float get(const T* p) { return __ldcg(p); }
    __device__ static void unpack(const uint32_t* w, float (&x)[16]) {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(w[i]);
    }
};
template <>
struct Elem<kDtBf16> {
    using T = unsigned short;
    static constexpr unsigned kNone = 0xFF80u;
    __device__ static T put(float x) { return (T)(__float_as_uint(x) >> 16); }
    __device__ static float at(T x) { return __uint_as_float((unsigned)x << 16); }
    __device__ static float get(const T* p) { return __uint_as_float((unsigned)__ldcg(p) << 16); }
    __device__ static void unpack(const uint32_t* w, float (&x)[16]) {
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
    __device__ static T put(float x) { return __half_as_ushort(__float2half_rn(x)); }
    __device__ static float at(T x) { return __half2float(__ushort_as_half(x)); }
    __device__ static float get(const T* p) { return __half2float(__ushort_as_half(__ldcg(p))); }
    __device__ static void unpack(const uint32_t* w, float (&x)[16]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
};

// 32 bytes from a 32-byte boundary, one whole sector, without a copy left in L1 or with one (where a neighbour reads the
// sector too); 16 bytes from a 16-byte boundary.
__device__ __forceinline__ void load_sector(const void* p, uint32_t* r) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "l"(p));
}
__device__ __forceinline__ void load_shared_sector(const void* p, uint32_t* r) {
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "l"(p));
}
__device__ __forceinline__ void load_half(const void* p, uint32_t* r) {
    asm volatile("ld.global.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "l"(p));
}

// A row's share: where it starts, and which of its units can be read in whole sectors.
template <int DT>
struct Share {
    using E = Elem<DT>;
    using T = typename E::T;
    static constexpr int kWords = kUnit * (int)sizeof(T) / 4;  // 32-bit words of a unit
    // A row that starts at no sector's start is read in pieces of this many bytes, shifted (a unit of 16-bit values is one
    // sector: in halves it takes 48 bytes instead of 64)
    static constexpr int kPiece = sizeof(T) == 4 ? 32 : 16;
    const T* p;      // first token of the share
    int len, units;  // tokens, units (the last may be partial)
    int lo, hi;      // units [lo, hi) are whole and the pieces they touch lie inside the tensor

    __device__ void set(const T* tensor, const T* tensor_end, const T* first, int n) {
        p = first;
        len = n;
        units = (n + kUnit - 1) / kUnit;
        hi = n / kUnit;
        lo = 0;
        const int off = (int)(reinterpret_cast<uintptr_t>(p) % kPiece);
        if (off) {  // a unit's pieces then start before it and end behind it, by less than one
            const char* c = reinterpret_cast<const char*>(p) - off;
            if (c < reinterpret_cast<const char*>(tensor)) lo = 1;
            if (hi > 0 && c + (size_t)hi * (kWords * 4) + kPiece > reinterpret_cast<const char*>(tensor_end)) --hi;
        }
    }
    // SHIFT: elements from the piece's boundary at or below p to p, the same for every unit; -1: p is at a sector's start.
    // What a unit of [lo, hi), at c, lies in; and its values as words from that.  The thread that holds a token, and so
    // the order of every sum, does not depend on where the row starts.
    template <int SHIFT>
    static constexpr int kHeld = kWords + (SHIFT > 0 ? kPiece / 4 : 0);
    template <int SHIFT>
    __device__ static void fetch(const char* c, uint32_t* raw) {
        if constexpr (SHIFT < 0) {
#pragma unroll
            for (int i = 0; i < kWords / 8; ++i) load_sector(c + 32 * i, raw + 8 * i);
        } else {
            c -= SHIFT * (int)sizeof(T);
#pragma unroll
            for (int i = 0; i < kHeld<SHIFT> * 4 / kPiece; ++i) {
                if constexpr (kPiece == 32) load_shared_sector(c + 32 * i, raw + 8 * i);
                else load_half(c + 16 * i, raw + 4 * i);
            }
        }
    }
    __device__ const char* unit(int u) const { return reinterpret_cast<const char*>(p) + (size_t)u * (kWords * 4); }
    template <int SHIFT>
    __device__ static void words(const uint32_t* raw, uint32_t* w) {
        constexpr int kFirst = SHIFT < 0 ? 0 : SHIFT * (int)sizeof(T) / 4;
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if constexpr (SHIFT > 0 && sizeof(T) == 2 && SHIFT % 2 == 1)
                w[i] = __funnelshift_r(raw[kFirst + i], raw[kFirst + i + 1], 16);
            else
                w[i] = raw[kFirst + i];
        }
    }
    // Unit u token by token, -inf behind the share's end: at the tensor's edges.
    __device__ void tokens(int u, uint32_t* w) const {
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
};

// A number as the unevaluated sum of two floats (48 bits): the 64-bit unit of this GPU takes some hundred cycles an
// operation.  two_sum and its use here are Knuth's error-free addition.
struct Two {
    float hi, lo;
};
__device__ __forceinline__ Two two_sum(float a, float b) {
    const float s = a + b, t = s - a;
    return Two{s, (a - (s - t)) + (b - t)};
}
__device__ __forceinline__ Two add(Two a, Two b) {
    const Two s = two_sum(a.hi, b.hi);
    const float lo = s.lo + (a.lo + b.lo), hi = s.hi + lo;
    return Two{hi, lo - (hi - s.hi)};
}
__device__ __forceinline__ Two warp_sum(Two v, int lanes) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        if (o >= lanes) break;
        v = add(v, Two{__shfl_xor_sync(0xffffffffu, v.hi, o), __shfl_xor_sync(0xffffffffu, v.lo, o)});
    }
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// How many of the n keys are above `key` (low half) and equal to it (high half), counted by LANES neighbouring
// threads together; every thread of the warp calls it, `sub` is the thread's number among the LANES.
template <int LANES>
__device__ __forceinline__ unsigned rank_of(const unsigned long long* keys, int n, unsigned long long key, int sub) {
    unsigned r = 0;
#pragma unroll 4
    for (int i = sub; i < n; i += LANES) {
        const unsigned long long k = keys[i];
        r += k > key ? 1u : (k == key ? 0x10000u : 0u);
    }
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
    return r;
}

// The best of a team of `team` neighbouring threads, and the number of teams ahead of this one (low half) and of equal
// best (high half); top: a word per team, written by one of it.
__device__ __forceinline__ unsigned long long team_best(unsigned long long v, int team) {
    unsigned long long y = __shfl_xor_sync(0xffffffffu, v, 1);
    v = y > v ? y : v;
    y = __shfl_xor_sync(0xffffffffu, v, 2);
    return team == 4 && y > v ? y : v;
}
__device__ __forceinline__ unsigned team_rank(const unsigned long long* top, unsigned long long key, int team, int lane) {
    return team == 4 ? rank_of<4>(top, kThreads / 4, key, lane & 3) : rank_of<2>(top, kThreads / 2, key, lane & 1);
}

// What a thread gathers on its way through a share: sum of 2^(x L - r2), the best group it met and its maximum.
struct Gather {
    float2 s2[2];
    float r2, best;
    int best_g;
};

// One unit's words: its group's maximum to gmax, its exponentials to the sums.
template <int DT>
__device__ __forceinline__ void take(const uint32_t* w, int u, bool store, typename Elem<DT>::T* gmax, Gather& t) {
    float x[kUnit];
    Elem<DT>::unpack(w, x);
    float m4[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) m4[i] = fmaxf(fmax3(x[4 * i], x[4 * i + 1], x[4 * i + 2]), x[4 * i + 3]);
    float gm = fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]);
    gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, 1));  // the other half of the group
    if (store) gmax[u >> 1] = Elem<DT>::put(gm);
    t.best_g = gm > t.best ? u >> 1 : t.best_g;
    t.best = fmaxf(t.best, gm);
    // sums up to 2^kSlack times the reference's lose nothing, so it moves once or twice a row, not with every new
    // maximum (in a warp, one thread or another meets one nearly every time)
    if (gm * kL > t.r2 + kSlack) {
        const float r = ceilf(gm * kL), f = pow2_down(t.r2 - r);
#pragma unroll
        for (int i = 0; i < 2; ++i) t.s2[i] = make_float2(t.s2[i].x * f, t.s2[i].y * f);
        t.r2 = r;
    }
    const float2 l2 = make_float2(kL, kL), neg = make_float2(-t.r2, -t.r2);
#pragma unroll
    for (int i = 0; i < kUnit / 2; ++i) {
        const float2 y = ffma2(make_float2(x[2 * i], x[2 * i + 1]), l2, neg);
        t.s2[i & 1] = fadd2(t.s2[i & 1], make_float2(fast_exp2(y.x), fast_exp2(y.y)));
    }
}

// One pass over the share.  A group is two neighbouring threads' units.
template <int DT, int SHIFT>
__device__ __forceinline__ void stream(const Share<DT>& sh, typename Elem<DT>::T* gmax, Gather& t) {
    using S = Share<DT>;
    constexpr int kWords = S::kWords, kHeld = S::template kHeld<SHIFT>;
    constexpr int kBatch = SHIFT < 0 ? 32 / kWords : (kWords == 16 ? 1 : 2);  // units loaded together
    const int tid = threadIdx.x;
    int u0 = tid;
    auto any = [&](int u, uint32_t* w) {  // any unit's words
        if (u >= sh.lo && u < sh.hi) {
            uint32_t raw[kHeld];
            S::template fetch<SHIFT>(sh.unit(u), raw);
            S::template words<SHIFT>(raw, w);
        } else if (u < sh.units) {
            sh.tokens(u, w);
        } else {
#pragma unroll
            for (int i = 0; i < kWords; ++i) w[i] = kWords == 16 ? Elem<DT>::kNone : Elem<DT>::kNone * 0x10001u;
        }
    };
    auto careful = [&]() {  // a step's units, whichever they are
        if constexpr (SHIFT < 0) {
            uint32_t w[kBatch][kWords];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) any(u0 + b * kThreads, w[b]);
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int u = u0 + b * kThreads;
                take<DT>(w[b], u, !(tid & 1) && u < sh.units, gmax, t);
            }
        } else {  // one at a time: the many shifted loops' code stays small
#pragma unroll 1
            for (int u = u0; u < u0 + kBatch * kThreads && u - (tid & 31) < sh.units; u += kThreads) {
                uint32_t w[kWords];
                any(u, w);
                take<DT>(w, u, !(tid & 1) && u < sh.units, gmax, t);
            }
        }
    };
    if (sh.lo) {
        careful();
        u0 += kThreads * kBatch;
    }
    const char* c = sh.unit(u0);
    // while the warps' units are whole: no tests
    for (; (u0 | 31) + (kBatch - 1) * kThreads < sh.hi; u0 += kThreads * kBatch, c += kThreads * kBatch * (kWords * 4)) {
        uint32_t raw[kBatch][kHeld];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) S::template fetch<SHIFT>(c + b * kThreads * (kWords * 4), raw[b]);
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            uint32_t w[kWords];
            S::template words<SHIFT>(raw[b], w);
            take<DT>(w, u0 + b * kThreads, !(tid & 1), gmax, t);
        }
    }
    for (; u0 - (tid & 31) < sh.units; u0 += kThreads * kBatch) careful();
}
// The same for where the share starts, which is known only now: one loop for each of the places that a row may start at (64 x
// 8 rows of 200001 bf16: 49 us; with the shift chosen at run time 60).
template <int DT, int SHIFT = 0>
__device__ __forceinline__ void stream_from(int shift, const Share<DT>& sh, typename Elem<DT>::T* gmax, Gather& t) {
    if constexpr (SHIFT < Share<DT>::kPiece / (int)sizeof(typename Elem<DT>::T)) {
        if (shift == SHIFT) stream<DT, SHIFT>(sh, gmax, t);
        else stream_from<DT, SHIFT + 1>(shift, sh, gmax, t);
    }
}

struct SelectSmem {
    alignas(16) unsigned long long top[kMaxTeams];  // the teams' best groups
    float s[kThreads], r[kThreads];              // the threads' sums and references
    int sel[kBeamMaxSelect];
    unsigned long long threshold;
    int found[3];  // entries of the lists of groups, of tokens and of the tokens that a second threshold leaves: a word
                   // each, so that none is written again while it may still be read
};
// Behind it: the groups at or above the threshold (M teams' at most), and every group's maximum, in the logits' type, which
// the tokens of the M best replace.  What is left of the SM's memory is L1, and the loads in flight want it: the 64 x 8
// rows of 200000 take 52 us with 60 KB of L1 and 42 with 124.
__host__ __device__ inline int groups_of(int tokens) { return (tokens + kGroup - 1) / kGroup; }
__host__ __device__ inline int list_cap(int groups, int M) {  // a team has at most two of every kThreads / 2 groups
    return M * 2 * ((groups + kThreads / 2 - 1) / (kThreads / 2));
}
inline size_t select_smem(int part_len, int M, int dtype) {
    const size_t groups = groups_of(part_len), maxima = ((groups + 3) & ~size_t(3)) * (dtype == kDtF32 ? 4 : 2);
    const size_t tokens = (size_t)M * kGroup * 8;
    return sizeof(SelectSmem) + (size_t)list_cap((int)groups, M) * 8 + (maxima > tokens ? maxima : tokens);
}

template <int DT>
__global__ void __launch_bounds__(kThreads, 4) select_rows_kernel(const BeamArgs a) {
    using E = Elem<DT>;
    using T = typename E::T;
    constexpr int kWords = Share<DT>::kWords;
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
    T* gmax = reinterpret_cast<T*>(tokens);

    // ---- 1. one pass over the share
    Gather t = {{make_float2(0.f, 0.f), make_float2(0.f, 0.f)}, -1e9f, kNegInf, 0};
    const unsigned start = (unsigned)reinterpret_cast<uintptr_t>(sh.p);
    if (start % 32 == 0) stream<DT, -1>(sh, gmax, t);
    else stream_from<DT>((int)(start % Share<DT>::kPiece / sizeof(T)), sh, gmax, t);
    sm.s[tid] = (t.s2[0].x + t.s2[0].y) + (t.s2[1].x + t.s2[1].y);
    sm.r[tid] = t.r2;
    unsigned long long top = t.best > kNegInf ? ((unsigned long long)ord32(t.best) << 32) | (unsigned)~t.best_g : 0ull;
    const int team = team_of(M), teams = kThreads / team;
    top = team_best(top, team);
    if (top == 0) top = (unsigned long long)(teams - 1 - tid / team);  // below every group, and different in every team
    if (tid % team == 0) sm.top[tid / team] = top;
    if (tid < 3) sm.found[tid] = 0;
    __syncthreads();

    // ---- 2. the share's maximum; its sum again against that maximum where it is far out
    float m_all;
    {
        unsigned o = 0;
        for (int i = lane; i < teams; i += 32) o = max(o, (unsigned)(sm.top[i] >> 32));
        o = __reduce_max_sync(0xffffffffu, o);
        m_all = o ? unord32(o) : kNegInf;
    }
    const bool far = m_all > kPlainRange || (m_all < -kPlainRange && m_all != kNegInf);
    if (far) {
        float sum = 0.f;
        for (int u = tid; u < sh.units; u += kThreads) {
            uint32_t w[kWords];
            float x[kUnit];
            sh.tokens(u, w);
            E::unpack(w, x);
#pragma unroll
            for (int i = 0; i < kUnit; ++i) sum += fast_exp2((x[i] - m_all) * kL);
        }
        sm.s[tid] = sum;
        __syncthreads();
    }

    // ---- 3. the threshold: the M-th best of the teams' best groups; meanwhile the last warp adds the sums up
    if ((team_rank(sm.top, top, team, lane) & 0xffffu) == (unsigned)(M - 1)) sm.threshold = top;  // the whole team
    // the last warp adds the threads' sums up meanwhile, a part of it in each of the next stages
    const bool adds = warp == kThreads / 32 - 1;
    float r_all = kNegInf;
    if (adds) {
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) r_all = fmaxf(r_all, sm.r[lane + 32 * i]);
        r_all = warp_max(r_all);
    }
    __syncthreads();
    const unsigned long long thr = sm.threshold;
    {
        const float thr_f = (thr >> 32) ? unord32((unsigned)(thr >> 32)) : kNegInf;
        for (int g0 = 4 * tid; g0 < groups; g0 += 4 * kThreads) {
            struct alignas(4 * sizeof(T)) Four {
                T x[4];
            };
            const Four four = *reinterpret_cast<const Four*>(gmax + g0);
            const float v[4] = {E::at(four.x[0]), E::at(four.x[1]), E::at(four.x[2]), E::at(four.x[3])};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (v[i] >= thr_f && v[i] > kNegInf && g0 + i < groups) {
                    const unsigned long long key = ((unsigned long long)ord32(v[i]) << 32) | (unsigned)~(g0 + i);
                    if (key >= thr) list[atomicAdd(&sm.found[0], 1)] = key;
                }
            }
        }
    }
    Two sum = {0.f, 0.f};
    if (adds) {
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) {  // scaled by exact powers of two (a NaN stays one)
            const float x = far ? sm.s[lane + 32 * i] : sm.s[lane + 32 * i] * pow2_down(sm.r[lane + 32 * i] - r_all);
            sum = add(sum, Two{x, 0.f});
        }
    }
    __syncthreads();
    const int n = sm.found[0];  // <= M x (groups of a team)
    for (int i0 = 0; i0 < n; i0 += kThreads / 8) {
        const int i = i0 + (tid >> 3);
        const unsigned long long key = i < n ? list[i] : 0ull;
        const int r = (int)(rank_of<8>(list, n, key, lane & 7) & 0xffffu);
        if (i < n && r < M) sm.sel[r] = (int)~(unsigned)key;
        if (i < n && r == M - 1) sm.threshold = key;  // M tokens are at least this group's best
    }
    if (adds) {
        sum = warp_sum(sum, 32);
        if (lane == 0) a.part[blockIdx.x] = BeamPart{far ? kInf : r_all, m_all, sum.hi, sum.lo};
    }
    __syncthreads();

    // ---- 4. the tokens of the best groups that can be among the M best, ranked
    const unsigned thr_v = (unsigned)(sm.threshold >> 32);
    for (int i = tid; i < min(n, M) * kGroup; i += kThreads) {
        const int e = sm.sel[i / kGroup] * kGroup + i % kGroup;
        if (e >= sh.len) continue;
        const float v = E::get(sh.p + e);
        const unsigned o = ord32(v);
        if (v > kNegInf && o >= thr_v)
            tokens[atomicAdd(&sm.found[1], 1)] = ((unsigned long long)o << 32) | (unsigned)~(e0 + e);
    }
    __syncthreads();
    int nt = sm.found[1];
    if (nt > kThreads) {
        // few groups, or many equal values: the M-th best of the teams' best tokens is a threshold again
        constexpr int kHeld = kBeamMaxSelect * kGroup / kThreads;
        unsigned long long held[kHeld], best = 0;
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            held[i] = tid + i * kThreads < nt ? tokens[tid + i * kThreads] : 0ull;
            best = held[i] > best ? held[i] : best;
        }
        best = team_best(best, team);  // every thread has one
        if (tid % team == 0) sm.top[tid / team] = best;
        __syncthreads();
        if ((team_rank(sm.top, best, team, lane) & 0xffffu) == (unsigned)(M - 1)) sm.threshold = best;
        __syncthreads();
        const unsigned long long least = sm.threshold;
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            if (held[i] && held[i] >= least) tokens[atomicAdd(&sm.found[2], 1)] = held[i];
        __syncthreads();
        nt = sm.found[2];
    }
    unsigned long long* out = a.best + (size_t)blockIdx.x * M;
    for (int i0 = 0; i0 < nt; i0 += kThreads / 8) {
        const int i = i0 + (tid >> 3);
        const unsigned long long key = i < nt ? tokens[i] : 0ull;
        const int r = (int)(rank_of<8>(tokens, nt, key, lane & 7) & 0xffffu);
        if (i < nt && r < M && (lane & 7) == 0) out[r] = key;
    }
    if (tid >= nt && tid < M) out[tid] = 0;
}

// ---------------------------------------------------------------------------- merge over a group's rows
// Order of a finite score hi + lo as an unsigned number; every score's is above 0.
__device__ __forceinline__ unsigned long long ord_two(Two x) {
    return ((unsigned long long)ord32(x.hi) << 32) | ord32(x.lo);
}
// ... and of c + (z - lse), all finite.  Where a sum on the way leaves f32's range (a mask of the type's lowest value on a beam
// marked by the lowest score) it is taken again in quarters, which stay inside; a score below the range is -inf, after all
// that are within it and among its like by the quarter as f32 holds it.
__device__ __forceinline__ unsigned long long ord_score(float c, float z, Two lse) {
    auto sum = [&](float f) {
        const Two d = two_sum(f * z, -f * lse.hi);
        return add(Two{f * c, 0.f}, Two{d.hi, d.lo - f * lse.lo});
    };
    const Two x = sum(1.f);
    if (fabsf(x.hi) < kInf) return ord_two(x);  // neither infinite nor, from two infinities, a NaN
    const Two q = sum(0.25f);
    if (fabsf(4.f * q.hi) < kInf) return ord_two(Two{4.f * q.hi, 4.f * q.lo});
    return ((unsigned long long)ord32(kNegInf) << 32) | ord32(q.hi);
}

// (r + log2 s) / kL for an integer r, a positive s = hi + lo and kL = L as rounded: to about 2e-9 of the logarithm.
// s = 2^e m with m in [sqrt(1/2), sqrt(2)), n = m - 1, and the series of ln m = 2 artanh t, t = n / (n + 2), |t| < 0.172,
// cut behind t^9 / 9 (the next term is below 4e-10); its leading terms carry a second float.  The products that a two_sum takes
// are rounded on their own (__fmul_rn): contracted into its additions they would be counted with two errors.
__device__ __forceinline__ Two natural_log(float r, Two s) {
    const int b = __float_as_int(s.hi);
    int e = (b >> 23) - 127;
    if ((b & 0x7fffff) > 0x3504f3) ++e;  // above sqrt(2): half of it
    const float scale = __int_as_float((127 - e) << 23);
    const float nh = s.hi * scale - 1.f, nl = s.lo * scale;  // exact
    const float den = nh + 2.f;
    const float th = __fdividef(nh, den);
    const float tl = __fdividef(fmaf(-th, nh, fmaf(-2.f, th, nh)) + nl * (1.f - th), den);
    const float q = th * th;
    float p = fmaf(q, 1.f / 9.f, 1.f / 7.f);
    p = fmaf(p, q, 1.f / 5.f);
    p = fmaf(p, q, 1.f / 3.f);
    constexpr float kCh = 2.885390043258667f;          // 2 / ln 2 as two floats
    constexpr float kCl = 3.8519259e-08f;
    const float ph = __fmul_rn(kCh, th);
    const float pl = fmaf(kCh, th, -ph) + (fmaf(kCh, tl, kCl * th) + ph * q * p);
    const Two l2 = add(two_sum(r + (float)e, ph), Two{pl, 0.f});
    constexpr double kInv = 1.0 / (double)kL;          // as two floats
    constexpr float kIh = (float)kInv, kIl = (float)(kInv - (double)kIh);
    const float h = __fmul_rn(l2.hi, kIh);
    return add(Two{h, fmaf(l2.hi, kIh, -h)}, Two{fmaf(l2.hi, kIl, l2.lo * kIh), 0.f});
}
__device__ __forceinline__ Two to_two(double x) {
    const float hi = (float)x;
    return Two{hi, (float)(x - (double)hi)};
}

struct MergeSmem {
    alignas(16) unsigned long long top[kMaxTeams];  // the teams' best scores' orders, 0: none
    Two lse[kBeamMaxBeams];
    float cum[kBeamMaxBeams];
    int state[kBeamMaxBeams];  // 0: no continuation, 1: read, 2: finished
    unsigned long long threshold;
    int found;
};
// Behind it: score order and (beam, token) of the K x parts x M candidates, then of those at or above the threshold.
inline size_t merge_smem(int total) { return sizeof(MergeSmem) + (size_t)((total + 1) & ~1) * 32; }

__global__ void __launch_bounds__(kThreads) select_merge_kernel(const BeamArgs a) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    MergeSmem& sm = *reinterpret_cast<MergeSmem*>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, n = blockIdx.x;
    const int K = a.K, M = a.M, parts = a.parts, shares = K * parts, total = shares * M;
    unsigned long long* score = reinterpret_cast<unsigned long long*>(&sm + 1);
    unsigned long long* at = score + ((total + 1) & ~1);
    unsigned long long* list_score = at + ((total + 1) & ~1);
    unsigned long long* list_at = list_score + ((total + 1) & ~1);
    if (tid == 0) sm.found = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // the first candidates are on their way while the rows' sums are put together (those of rows that were not read
    // hold anything and are not looked at)
    constexpr int kAhead = 4;
    const unsigned long long* best = a.best + (long long)n * total;
    // Which candidate is the i-th, so that the best are spread over the teams (where they meet in a few, the threshold is low).
    // Few shares: their best ones, then their second and so on (26 groups of 16 rows, 24 picks: 12.5 us, 13.7 share by share).
    // Many: share by share, which reads in lines (8 groups of 8 rows of four shares: 13.5 us, 14.6 rank by rank).  Many picks:
    // share by share, each turned by one more than the one before (32 beams, 64 picks: 25 us, 40 rank by rank).
    const bool by_rank = M <= 32 && parts <= 2;
    auto share_at = [&](int i) { return by_rank ? i % shares : i / M; };
    auto rank_at = [&](int i, int share) { return by_rank ? i / shares : (i - share * M + (M > 32 ? share : 0)) % M; };
    auto load = [&](int i) { return __ldcg(&best[share_at(i) * M + rank_at(i, share_at(i))]); };
    unsigned long long ahead[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) ahead[j] = tid + j * kThreads < total ? load(tid + j * kThreads) : 0ull;

    // ---- 1. each row's log-sum-exp from its shares: 8, 16 or 32 lanes a row, a lane per share
    const int lanes = parts <= 8 ? 8 : (parts <= 16 ? 16 : 32), sub = tid & (lanes - 1);
    for (int k0 = 0; k0 < K; k0 += kThreads / lanes) {  // whole warps: what is found of a row is in all its lanes
        const int k = k0 + tid / lanes, there = k < K ? parts : 0;
        const long long row = (long long)n * K + (k < K ? k : 0);
        const float c = __ldcg(&a.scores[row]);
        const bool done = a.finished && __ldcg(&a.finished[row]);
        const float4* p = reinterpret_cast<const float4*>(a.part + row * parts);
        const float4 own = sub < there ? __ldcg(p + sub) : make_float4(0.f, 0.f, 0.f, 0.f);
        auto get = [&](int i) { return i == sub ? own : __ldcg(p + i); };
        float m = kNegInf, r = -1e9f, flags = 0.f;  // flags: 1 far out, 2 NaN
        for (int i = sub; i < there; i += lanes) {
            const float4 x = get(i);
            m = fmaxf(m, x.y);
            r = x.x == kInf ? r : fmaxf(r, x.x);
            flags = fmaxf(flags, x.z != x.z ? 2.f : (x.x == kInf ? 1.f : 0.f));
        }
        for (int o = 1; o < lanes; o <<= 1) {
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            r = fmaxf(r, __shfl_xor_sync(0xffffffffu, r, o));
            flags = fmaxf(flags, __shfl_xor_sync(0xffffffffu, flags, o));
        }
        Two sum = {0.f, 0.f};
        for (int i = sub; i < there; i += lanes) {
            const float4 x = get(i);
            const float f = pow2_down(x.x - r);
            sum = add(sum, Two{x.z * f, x.w * f});
        }
        sum = warp_sum(sum, lanes);
        int st = c > kNegInf && c < kInf ? (done ? 2 : 1) : 0;
        bool bad = k < K && (c != c || c == kInf);
        Two l = {0.f, 0.f};
        if (st == 1) {
            if (flags == 2.f || m == kInf) {
                bad = k < K;
                st = 0;
            } else if (m == kNegInf) {  // every token is masked
                st = 0;
            } else {
                l = natural_log(r, sum);
            }
        }
        if (__any_sync(0xffffffffu, flags == 1.f && st == 1)) {  // shares far out: in 64 bits
            double d = 0.0;
            for (int i = sub; i < there; i += lanes) {
                const float4 x = get(i);
                if (x.y == kNegInf) continue;
                const double s = (double)x.z + (double)x.w;
                const double li = x.x == kInf ? (double)x.y + log(s) : ((double)x.x + log2(s)) / (double)kL;
                d += exp(li - (double)m);
            }
            for (int o = 1; o < lanes; o <<= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
            if (flags == 1.f && st == 1) l = to_two((double)m + log(d));
        }
        if (sub == 0 && k < K) {
            if (bad) atomicOr(a.err, kErrBadValue);
            sm.lse[k] = l;
            sm.cum[k] = c;
            sm.state[k] = st;
        }
    }
    __syncthreads();

    // ---- 2. the candidates; the M-th best of the teams' best scores bounds the M-th best of all
    unsigned long long mine = 0;
    int j = 0;
#pragma unroll 1
    for (int i = tid; i < total; i += kThreads, ++j) {
        unsigned long long key = ahead[0], x = 0, where = 0;
        if (j < kAhead) {
#pragma unroll
            for (int q = 1; q < kAhead; ++q) key = j == q ? ahead[q] : key;
        } else {
            key = load(i);
        }
        const int share = share_at(i), k = share / parts, st = sm.state[k];
        if (st == 1 && key) {
            x = ord_score(sm.cum[k], unord32((unsigned)(key >> 32)), sm.lse[k]);
            where = ((unsigned long long)k << 32) | ~(unsigned)key;
        } else if (st == 2 && share == k * parts && rank_at(i, share) == 0) {
            x = ord_two(Two{sm.cum[k], 0.f});
            where = ((unsigned long long)k << 32) | (unsigned)a.pad_token;
        }
        score[i] = x;
        at[i] = where;
        mine = x > mine ? x : mine;
    }
    const unsigned long long own = mine;
    const int team = team_of(M);
    mine = team_best(mine, team);
    if (tid % team == 0) sm.top[tid / team] = mine;
    __syncthreads();
    {
        const unsigned r = team_rank(sm.top, mine, team, lane), above = r & 0xffffu, level = r >> 16;
        if (above < (unsigned)M && above + level >= (unsigned)M) sm.threshold = mine;  // equal scores write the same
    }
    __syncthreads();
    const unsigned long long thr = sm.threshold;
    if (own && own >= thr) {
        for (int i = tid; i < total; i += kThreads) {
            const unsigned long long x = score[i];
            if (x && x >= thr) {
                const int to = atomicAdd(&sm.found, 1);
                list_score[to] = x;
                list_at[to] = at[i];
            }
        }
    }
    __syncthreads();

    // ---- 3. ranked by counting; equal scores by beam and token
    const int found = sm.found;
    for (int i0 = 0; i0 < found; i0 += kThreads / 8) {
        const int i = i0 + (tid >> 3);
        const unsigned long long x = i < found ? list_score[i] : 0ull, where = i < found ? list_at[i] : 0ull;
        int q = 0;
#pragma unroll 4
        for (int o = lane & 7; o < found; o += 8)
            q += (list_score[o] > x) | ((list_score[o] == x) & (list_at[o] < where));
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
        if (i >= found || (lane & 7) != 0) continue;
        if (q < M) {
            a.out_scores[(long long)n * M + q] = unord32((unsigned)(x >> 32));
            a.out_parents[(long long)n * M + q] = n * K + (int)(where >> 32);
            a.out_tokens[(long long)n * M + q] = (int)(unsigned)where;
        }
    }
    if (tid >= found && tid < M) {
        a.out_scores[(long long)n * M + tid] = kNegInf;
        a.out_parents[(long long)n * M + tid] = -1;
        a.out_tokens[(long long)n * M + tid] = -1;
    }
}

// Lets the four kernels have the shared memory that any call may ask for, once per device and thread.  The limits belong to the
// process: every thread sets the same ones, whatever its own call needs, so none is lowered under another's call.
cudaError_t allow_smem() {
    static thread_local bool allowed[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && allowed[dev])) return e;
    auto allow = [](const void* kernel, size_t bytes) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    };
    constexpr int M = kBeamMaxSelect;
    const void* rows[3] = {reinterpret_cast<const void*>(select_rows_kernel<kDtF32>),
                           reinterpret_cast<const void*>(select_rows_kernel<kDtBf16>),
                           reinterpret_cast<const void*>(select_rows_kernel<kDtF16>)};
    const int types[3] = {kDtF32, kDtBf16, kDtF16};
    for (int i = 0; i < 3; ++i)
        if ((e = allow(rows[i], select_smem(kBeamMaxPart, M, types[i]))) != cudaSuccess) return e;
    if ((e = allow(reinterpret_cast<const void*>(select_merge_kernel), merge_smem(kBeamMaxCands))) != cudaSuccess) return e;
    if (dev < 64) allowed[dev] = true;
    return cudaSuccess;
}

}  // namespace

cudaError_t beam_plan(int N, int K, int V, int M, BeamPlan* plan) {
    int sms = 0, dev = 0;
    cudaError_t e;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    const long long rows = (long long)N * K;
    // shares of a row: as many as run at once (four CTAs an SM), but none below 4096 tokens (one step of a thread), and no
    // more than 512 candidates for the merge (8 groups of 8 rows of 200000, 16 picks: 13.5 us with 512 of them, 18 with 1024),
    // or 768 where the SMs would not even be half full (5 groups of 12 rows of 143530, 23 picks: 17.3 us, 23.8 with one share a row)
    long long parts = rows > 0 ? (4ll * sms) / rows : 1;
    const long long fine = V / 4096;
    if (parts > fine) parts = fine;
    const long long least = ((long long)V + kBeamMaxPart - 1) / kBeamMaxPart;
    long long few = 512 / ((long long)K * M);
    if (2 * rows * few <= sms) few = 768 / ((long long)K * M);
    if (parts > few) parts = few;
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
    cfg.dynamicSmemBytes = select_smem(a.part_len, a.M, a.dtype);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void (*rows)(const BeamArgs) = a.dtype == kDtF32    ? select_rows_kernel<kDtF32>
                                   : a.dtype == kDtBf16 ? select_rows_kernel<kDtBf16>
                                                        : select_rows_kernel<kDtF16>;
    cudaError_t e = allow_smem();
    if (e != cudaSuccess) return e;
    if ((e = cudaLaunchKernelEx(&cfg, rows, a)) != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)a.N);
    cfg.dynamicSmemBytes = merge_smem(a.K * a.parts * a.M);
    return cudaLaunchKernelEx(&cfg, select_merge_kernel, a);
}

}  // namespace sinkattn
