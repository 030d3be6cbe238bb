// sample.cu -- the next token of each row from its logits and a random number: temperature, top-k, top-p and min-p.
//
// With m the row's largest logit and w(z) = e^((z - m) / t) a logit's weight, tokens are ordered by falling logit, equal ones by
// rising index.  top-k keeps the first k, top-p the shortest start of those whose weights reach p of their sum, min-p those with
// w >= min_p.  What is kept is always {z > z*} and the first r tokens with z = z*, so a row is a search for (z*, r) and then for the first
// token, in index order, at which the sum of the kept weights passes u Z.  Nothing is sorted.
//
// A row belongs to a cluster of up to eight CTAs that hold it in shared memory: the logits are read from HBM once, every later pass
// reads shared memory (what does not fit there is read again through L2).
//  * top-k's border is found by counting: the logits in 1024 bins of (z - m) / t, then, within the bin that holds the border, by their
//    bits as ordered integers, 1024 to a step, until a bin is one value.  Whole numbers: exact, the same in any order of the atomics, and
//    as good for ties (16-bit logits have thousands) as for none.  Where at most 1024 tokens can stay at all (as most rows have it),
//    they are listed after the first bins instead, sorted, and both borders read off one running sum.
//  * top-p's border is a place in a running sum of weights.  The counts, times the weight in a bin's middle, tell about where; the
//    weights above that are summed token by token, and those sums, with the sorted tokens or the counts of single values below,
//    decide.  A wrong guess is seen in the sums and corrected, never used.
//  * A token is picked by comparing sums over as many as 10^5 tokens whose weights are 10^-6 of the total each: sums in 32 bits (6e-8)
//    would pick another than exact arithmetic in a few rows of a thousand.  Sums are held in two floats (46 bits) and weights to
//    2^-28.5 (sample_weights.h): 2^y = 2^n 2^(i/32) 2^r, the middle factor in two floats from a table held by a warp's lanes, the last a
//    polynomial.  Errors of different logits mostly cancel, those of equal ones do not.  (64-bit arithmetic runs at 1/64 of the 32-bit
//    rate here.  Weights carried to 2^-38 cost 1.6 times as much: 127 us for the largest case below.)
//  * Sums are kept by warp; each warp owns a run of the row in index order, so the token's place is found among at most 64 runs, then
//    in one of them.  Kept ties need no list: the kept weights up to a token are (those with z > z*) + w(z*) min(r, number of
//    z = z* so far).
//
// Bound by neither HBM, which the row's one reading leaves idle 93% of the time and more, nor by one unit of the SM: at 80 registers and
// 74 KB three CTAs share an SM, whose issue slots are 35 to 37% busy; the rest are waits, on the instruction before, at barriers and on
// the cluster.  Measured (GB300): 256 rows of 50021 f32, settings of their own, 96 us (7.6 of reading): a CTA takes 27 us (load 2.3, maximum 2,
// first bins 5, list and sort 8 to 12, sums 2.5, the rest waits of eight exchanges within the cluster), 1024 CTAs in three waves; 64 rows
// of 200000 bf16, top-p of a flat distribution, 93 us (3.8): weights of every token twice, two waves.  One row of 32000: 15 to 19 us by its
// settings, latency.  f32 rows of 200000 leave one CTA on an SM (a chunk takes 100 KB): 64 of them 88 us without filters, 226 with top-p.
// Three CTAs an SM (80 registers) instead of two: 10% faster.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "args_sample.h"
#include "errors_beam.h"
#include "ptx.cuh"
#include "sample_sums.h"
#include "sample_weights.h"
#include "smem_limit.h"

namespace sinkattn {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 1024;
constexpr float kBinsPerOctave = 32.f;  // first bins: 32 to a factor of two of the weight
constexpr float kNegInf = -__builtin_huge_valf();
constexpr int kBatch = 64;              // steps of a run whose sums are held at a time while a token is looked for
constexpr int kList = 192;              // candidates of a warp's run that are kept apart
constexpr int kSort = 1024;             // candidates of a row that are sorted
static_assert(kSort <= kBins, "the sorted keys take the counts' place");


struct __align__(16) Smem {
    unsigned hist[kBins];  // this CTA's counts
    unsigned tot[kBins];   // the row's
    float seg[2][5][kMaxCluster * kWarps];  // what the warps of the row last shared: two sums of two floats and a count
    float2 scan_p[kWarps];
    unsigned scan_u[kWarps];
    float scan_f[kWarps];
    float2 step_a[kBatch];
    unsigned step_t[kBatch];
    int found, found_prev, found_next;
    unsigned found_count;
    float2 found_mass;
    float cutoff;
    int list_n[kWarps];             // candidates of each run; -1: not listed
    float list_z[kWarps][kList];
    int list_at[kWarps][kList];     // their places in the chunk
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address, in CTA `rank`'s shared memory, of what is at `p` in this one's.
__device__ __forceinline__ uint32_t remote(const void* p, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ void st_remote(uint32_t at, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_remote(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ float2 fmul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 neg2(float2 x) { return make_float2(-x.x, -x.y); }
// a + b = s + e exactly.
__device__ __forceinline__ float2 two_sum(float2 a, float2 b, float2& e) {
    const float2 s = fadd2(a, b), t = fadd2(s, neg2(a));
    e = fadd2(fadd2(a, neg2(fadd2(s, neg2(t)))), fadd2(b, neg2(t)));
    return s;
}

// ---------------------------------------------------------------- logits of each type: words of 16 bytes, ordered integer keys
template <typename T>
struct Logits;
template <>
struct Logits<float> {
    static constexpr int kPer = 4, kDrop = 0;
    static __device__ __forceinline__ void floats(uint4 w, float (&z)[4]) {
        z[0] = __uint_as_float(w.x), z[1] = __uint_as_float(w.y), z[2] = __uint_as_float(w.z), z[3] = __uint_as_float(w.w);
    }
};
template <>
struct Logits<__nv_bfloat16> {
    static constexpr int kPer = 8, kDrop = 16;
    static __device__ __forceinline__ void floats(uint4 w, float (&z)[8]) {
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            z[2 * i] = __uint_as_float(x[i] << 16);
            z[2 * i + 1] = __uint_as_float(x[i] & 0xFFFF0000u);
        }
    }
};
template <>
struct Logits<__half> {
    static constexpr int kPer = 8, kDrop = 13;
    static __device__ __forceinline__ void floats(uint4 w, float (&z)[8]) {
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x[i]));
            z[2 * i] = f.x;
            z[2 * i + 1] = f.y;
        }
    }
};

// A logit as an integer of the same order, without the low bits that its type leaves at zero (-0 counts as 0).
template <int kDrop>
__device__ __forceinline__ uint32_t key_of(float z) {
    const uint32_t b = __float_as_uint(z + 0.f);
    return ((b >> 31) ? ~b : b | 0x80000000u) >> kDrop;
}
template <int kDrop>
__device__ __forceinline__ float of_key(uint32_t k) {
    const uint32_t low = kDrop ? (1u << kDrop) - 1u : 0u;
    const uint32_t f = k << kDrop;
    return __uint_as_float((f >> 31) ? f & 0x7FFFFFFFu : ~(f | low));
}

// A bound b with z > b exactly where the key of z is above k, and z <= b where it is not.  (No logit has the key below zero's, which
// reads as -0 and would count with zero.)
template <int kDrop>
__device__ __forceinline__ float bound_of(uint32_t k) {
    const float z = of_key<kDrop>(k);
    return z == 0.f && (__float_as_uint(z) >> 31) ? __uint_as_float(0x80000001u) : z;
}

// ---------------------------------------------------------------- sums in two floats, within a warp
__device__ __forceinline__ double value(Pair a) { return (double)a.h + (double)a.l; }
__device__ __forceinline__ Pair shfl_up(Pair a, int o) {
    return {__shfl_up_sync(0xffffffffu, a.h, o), __shfl_up_sync(0xffffffffu, a.l, o)};
}
__device__ __forceinline__ unsigned shfl_up(unsigned a, int o) { return __shfl_up_sync(0xffffffffu, a, o); }
__device__ __forceinline__ float shfl_up(float a, int o) { return __shfl_up_sync(0xffffffffu, a, o); }
__device__ __forceinline__ Pair warp_sum(Pair a) {
#pragma unroll
    for (int o = 16; o; o >>= 1) a = a + Pair{__shfl_xor_sync(0xffffffffu, a.h, o), __shfl_xor_sync(0xffffffffu, a.l, o)};
    return a;
}
// Sum of x over the lanes below this one.
template <typename V>
__device__ __forceinline__ V lanes_below(V x, int lane) {
    V incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const V y = shfl_up(incl, o);
        if (lane >= o) incl = incl + y;
    }
    const V below = shfl_up(incl, 1);
    return lane ? below : V{};
}

// ---------------------------------------------------------------- weights
__device__ const float2 kRoots[32] = SINKATTN_ROOTS;

// Two numbers at a time.
struct TwoByTwo {
    using F = float2;
    static __device__ __forceinline__ F all(float x) { return make_float2(x, x); }
    static __device__ __forceinline__ F add(F a, F b) { return fadd2(a, b); }
    static __device__ __forceinline__ F mul(F a, F b) { return fmul2(a, b); }
    static __device__ __forceinline__ F fma(F a, F b, F c) { return ffma2(a, b, c); }
};

struct Weight : RowScale {
    float th, tl;  // this lane's entry of the table: 2^(lane / 32) in two floats
};

// Weights of two logits, each as hi + lo with lo at most half a step of hi; every lane of the warp calls.
__device__ __forceinline__ float2 weights2(const Weight& g, float2 z, float2& lo) {
    float2 y, k, r, h, l;
    split_power<TwoByTwo>(g, z, y, k, r);
    const int k0 = __float_as_int(k.x) - 0x4B400000, k1 = __float_as_int(k.y) - 0x4B400000;
    const float2 th = make_float2(__shfl_sync(0xffffffffu, g.th, k0 & 31), __shfl_sync(0xffffffffu, g.th, k1 & 31));
    const float2 tl = make_float2(__shfl_sync(0xffffffffu, g.tl, k0 & 31), __shfl_sync(0xffffffffu, g.tl, k1 & 31));
    root_times_power<TwoByTwo>(th, tl, r, h, l);
    // times 2^n
    const bool in0 = y.x > g.least, in1 = y.y > g.least;
    const int bias = 127 - g.base;
    const float2 s = make_float2(in0 ? __int_as_float(((k0 >> 5) + bias) << 23) : 0.f, in1 ? __int_as_float(((k1 >> 5) + bias) << 23) : 0.f);
    lo = make_float2(in0 ? l.x * s.x : 0.f, in1 ? l.y * s.y : 0.f);
    return make_float2(in0 ? h.x * s.x : 0.f, in1 ? h.y * s.y : 0.f);
}
// The weight of one logit a lane; all lanes call.
__device__ __forceinline__ Pair weight1(const Weight& g, float z) {
    float2 lo;
    const float2 hi = weights2(g, make_float2(z, z), lo);
    return {hi.x, lo.x};
}

// A first bin: falls with the logit, monotone because both roundings are, and 0 for the largest whatever its size (c32:
// -32 log2(e) / t).
__device__ __forceinline__ int bin_of(float z, float m, float c32) {
    return (int)min(__float2uint_rz(__fmul_rn(__fsub_rn(z, m), c32)), (unsigned)(kBins - 1));
}

// One row, as the threads of its cluster see it.
template <typename T>
struct Row {
    using L = Logits<T>;
    static constexpr int kPer = L::kPer, kDrop = L::kDrop;
    static constexpr uint32_t kNone = 0x007FFFFFu >> kDrop;  // the key of -inf; all that counts is above

    const T* chunk;     // this CTA's first logit
    const uint4* held;  // its words in shared memory
    int len, mis;       // logits of this CTA; how far its first lies behind a 16-byte boundary
    int resident;
    int w0, w1;         // this warp's words
    Smem* sm;
    uint32_t rank, size;
    int lane, warp, tid, turn;
    // Once few tokens are left their logits stand in a list for each run, which later passes read instead of the chunk: those with
    // keys in [list_lo, list_hi], where list_lo <= list_hi.
    uint32_t list_lo, list_hi;

    // Word w of this CTA's: kPer logits, -inf outside the chunk.
    __device__ __forceinline__ uint4 load(int w) const {
        const int e0 = w * kPer - mis;
        if (e0 >= 0 && e0 + kPer <= len) {
            uint4 x;
            asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                         : "l"(chunk + e0));
            return x;
        }
        union {
            uint4 v;
            T t[kPer];
        } u;
#pragma unroll
        for (int i = 0; i < kPer; ++i) u.t[i] = e0 + i >= 0 && e0 + i < len ? chunk[e0 + i] : (T)kNegInf;
        return u.v;
    }
    // Step `it` of this warp's run (or of run [a, b)): each lane's kPer logits, -inf behind the end.
    __device__ __forceinline__ void step(int a, int b, int it, float (&z)[kPer]) const {
        const int w = a + it * 32 + lane;
        if (w < b) {
            L::floats(w < resident ? held[w] : load(w), z);
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i) z[i] = kNegInf;
        }
    }
    __device__ __forceinline__ int steps() const { return (max(w1 - w0, 0) + 31) / 32; }
    // Whether this run's list (or run w's) holds all tokens with keys in [lo, hi]; its steps, and each lane's kPer of a step.
    __device__ __forceinline__ bool listed(uint32_t lo, uint32_t hi, int w) const {
        return list_lo <= lo && hi <= list_hi && sm->list_n[w] >= 0;
    }
    __device__ __forceinline__ int list_steps(int w) const { return (sm->list_n[w] + 32 * kPer - 1) / (32 * kPer); }
    __device__ __forceinline__ void list_step(int w, int it, float (&z)[kPer]) const {
        const int j = (it * 32 + lane) * kPer, n = sm->list_n[w];
#pragma unroll
        for (int i = 0; i < kPer; ++i) z[i] = j + i < n ? sm->list_z[w][j + i] : kNegInf;
    }
    // Lists the tokens with keys in [lo, hi], in index order, where they are few enough.
    __device__ void make_list(uint32_t lo, uint32_t hi) {
        const float zlo = of_key<kDrop>(lo), zhi = hi == 0xFFFFFFFFu ? -kNegInf : bound_of<kDrop>(hi);
        int n = 0;
        for (int it = 0, end = steps(); it < end && n <= kList; ++it) {
            float z[kPer];
            step(w0, w1, it, z);
            int mine = 0;
#pragma unroll
            for (int i = 0; i < kPer; ++i) mine += z[i] >= zlo && z[i] <= zhi;
            if (!__any_sync(0xffffffffu, mine)) continue;
            int at = n + (int)lanes_below((unsigned)mine, lane);
            n += (int)__reduce_add_sync(0xffffffffu, (unsigned)mine);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                if (z[i] >= zlo && z[i] <= zhi) {
                    if (at < kList) {
                        sm->list_z[warp][at] = z[i];
                        sm->list_at[warp][at] = token(w0 + it * 32 + lane, i);
                    }
                    ++at;
                }
            }
        }
        if (lane == 0) sm->list_n[warp] = n <= kList ? n : -1;
        list_lo = lo;
        list_hi = hi;
        __syncthreads();  // (another warp may read the list while the token is looked for)
    }
    __device__ __forceinline__ int token(int w, int i) const { return w * kPer - mis + i; }  // within the chunk

    // Counts the keys in [klo, khi] by (khi - key) >> shift (or, first, all by bin_of) and brings the row's counts to sm->tot.
    __device__ void clear_hist() {
        for (int i = tid; i < kBins; i += kThreads) sm->hist[i] = 0;
        __syncthreads();
    }
    __device__ void merge_hist() {
        cluster_sync();  // every CTA's counts are complete (and sm->tot is no longer read)
        const int per = kBins / (int)size;
        for (int i = tid; i < per; i += kThreads) {
            const int bin = (int)rank * per + i;
            unsigned s = 0;
            for (uint32_t c = 0; c < size; ++c) s += ld_remote(remote(&sm->hist[bin], c));
            for (uint32_t c = 0; c < size; ++c) st_remote(remote(&sm->tot[bin], c), s);
        }
        cluster_sync();
    }
    __device__ void count_bins(float m, float c32) {
        clear_hist();
        for (int it = 0, n = steps(); it < n; ++it) {
            float z[kPer];
            step(w0, w1, it, z);
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (z[i] > kNegInf) atomicAdd(&sm->hist[bin_of(z[i], m, c32)], 1u);
        }
        merge_hist();
    }
    __device__ void count_keys(uint32_t klo, uint32_t khi, int shift) {
        clear_hist();
        const bool list = listed(klo, khi, warp);
        const float zlo = of_key<kDrop>(klo), zhi = bound_of<kDrop>(khi);  // keys in [klo, khi]: -0 as the lower one is zero's
        for (int it = 0, n = list ? list_steps(warp) : steps(); it < n; ++it) {
            float z[kPer];
            if (list) list_step(warp, it, z);
            else step(w0, w1, it, z);
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (z[i] >= zlo && z[i] <= zhi) atomicAdd(&sm->hist[(khi - key_of<kDrop>(z[i])) >> shift], 1u);
        }
        merge_hist();
    }

    // The weights of a lane's logits with take(logit), added to (hi, lo); all lanes of the warp call.
    template <typename Take>
    static __device__ __forceinline__ void add_weights(const Weight& g, const float (&z)[kPer], Take take, float2& hi, float2& lo) {
#pragma unroll
        for (int i = 0; i < kPer; i += 2) {
            float2 vl, e;
            const float2 v = weights2(g, make_float2(z[i], z[i + 1]), vl);
            const bool t0 = take(z[i]), t1 = take(z[i + 1]);
            hi = two_sum(hi, make_float2(t0 ? v.x : 0.f, t1 ? v.y : 0.f), e);
            lo = fadd2(lo, fadd2(e, make_float2(t0 ? vl.x : 0.f, t1 ? vl.y : 0.f)));
        }
    }
    static __device__ __forceinline__ Pair joined(float2 hi, float2 lo) { return Pair{hi.x, lo.x} + Pair{hi.y, lo.y}; }

    // This warp's sum of the weights of keys in (klo, khi], and the number of keys equal to klo; in every lane.
    __device__ Pair sum(const Weight& g, uint32_t klo, uint32_t khi, unsigned& ties) {
        float2 hi = both(0.f), lo = both(0.f);
        unsigned n_ties = 0;
        const bool list = listed(klo, khi, warp);
        const float zlo = bound_of<kDrop>(klo), zhi = khi == 0xFFFFFFFFu ? -kNegInf : bound_of<kDrop>(khi);
        for (int it = 0, n = list ? list_steps(warp) : steps(); it < n; ++it) {
            float z[kPer];
            if (list) list_step(warp, it, z);
            else step(w0, w1, it, z);
            bool any = false;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                n_ties += z[i] == zlo;
                any |= z[i] > zlo && z[i] <= zhi;
            }
            if (!__any_sync(0xffffffffu, any)) continue;
            add_weights(g, z, [&](float x) { return x > zlo && x <= zhi; }, hi, lo);
        }
        ties = __reduce_add_sync(0xffffffffu, n_ties);
        return warp_sum(joined(hi, lo));
    }
    // The sums of the weights of keys above `at` and of those in (klo, at], and the counts of keys in [wlo, at] (as count_keys), in one
    // pass.
    __device__ void sum_apart(const Weight& g, uint32_t klo, uint32_t at, uint32_t wlo, int shift, Pair& above, Pair& rest) {
        clear_hist();
        const float zwlo = of_key<kDrop>(wlo);
        float2 hi = both(0.f), lo = both(0.f), rh = both(0.f), rl = both(0.f);
        const bool list = listed(klo + 1u, 0xFFFFFFFFu, warp);
        const float zlo = bound_of<kDrop>(klo), zat = bound_of<kDrop>(at);
        for (int it = 0, n = list ? list_steps(warp) : steps(); it < n; ++it) {
            float z[kPer];
            if (list) list_step(warp, it, z);
            else step(w0, w1, it, z);
            bool any = false;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                any |= z[i] > zlo;
                if (z[i] >= zwlo && z[i] <= zat) atomicAdd(&sm->hist[(at - key_of<kDrop>(z[i])) >> shift], 1u);
            }
            if (!__any_sync(0xffffffffu, any)) continue;
#pragma unroll
            for (int i = 0; i < kPer; i += 2) {
                float2 vl, e;
                const float2 v = weights2(g, make_float2(z[i], z[i + 1]), vl);
                const bool a0 = z[i] > zat, a1 = z[i + 1] > zat, r0 = !a0 && z[i] > zlo, r1 = !a1 && z[i + 1] > zlo;
                hi = two_sum(hi, make_float2(a0 ? v.x : 0.f, a1 ? v.y : 0.f), e);
                lo = fadd2(lo, fadd2(e, make_float2(a0 ? vl.x : 0.f, a1 ? vl.y : 0.f)));
                rh = two_sum(rh, make_float2(r0 ? v.x : 0.f, r1 ? v.y : 0.f), e);
                rl = fadd2(rl, fadd2(e, make_float2(r0 ? vl.x : 0.f, r1 ? vl.y : 0.f)));
            }
        }
        above = warp_sum(joined(hi, lo));
        rest = warp_sum(joined(rh, rl));
        merge_hist();
    }

    // The keys of all runs' lists, in falling order, in sm->hist of every CTA; false (in all) where a run has no list.  n: their number.
    __device__ bool sort_lists(int& n) {
        const int mine = sm->list_n[warp];
        const int s = share(Pair{0.f, 0.f}, Pair{0.f, 0.f}, (unsigned)mine);
        const int run = (int)rank * kWarps + warp, runs = (int)size * kWarps;
        unsigned c0 = shared_count(s, lane), c1 = lane + 32 < runs ? shared_count(s, lane + 32) : 0u;
        if (__any_sync(0xffffffffu, c0 == 0xFFFFFFFFu || c1 == 0xFFFFFFFFu)) return false;
        const unsigned at = __reduce_add_sync(0xffffffffu, (lane < run ? c0 : 0u) + (lane + 32 < run ? c1 : 0u));
        n = (int)__reduce_add_sync(0xffffffffu, c0 + c1);
        if (n > kSort) return false;
        for (int i = lane; i < mine; i += 32) {
            const uint32_t k = key_of<kDrop>(sm->list_z[warp][i]);
            for (uint32_t c = 0; c < size; ++c) st_remote(remote(&sm->hist[at + i], c), k);
        }
        int room = 32;
        while (room < n) room *= 2;
        for (int i = n + tid; i < room; i += kThreads) sm->hist[i] = 0;
        cluster_sync();
        for (int len = 2; len <= room; len *= 2)
            for (int gap = len / 2; gap; gap /= 2) {
                for (int i = tid; i < room / 2; i += kThreads) {
                    const int x = 2 * gap * (i / gap) + i % gap, y = x + gap;
                    const uint32_t kx = sm->hist[x], ky = sm->hist[y];
                    if ((kx < ky) == ((x & len) == 0)) {
                        sm->hist[x] = ky;
                        sm->hist[y] = kx;
                    }
                }
                __syncthreads();
            }
        return true;
    }

    // Every warp's sums to every CTA of the cluster: sm->seg[turn], by run in index order.  Returned: which of the two.
    __device__ int share(Pair a, Pair rest, unsigned n) {
        const int t = turn;
        turn ^= 1;
        if (lane < (int)size) {
            const uint32_t x[5] = {__float_as_uint(a.h), __float_as_uint(a.l), __float_as_uint(rest.h), __float_as_uint(rest.l), n};
#pragma unroll
            for (int i = 0; i < 5; ++i) st_remote(remote(&sm->seg[t][i][rank * kWarps + warp], lane), x[i]);
        }
        cluster_sync();
        return t;
    }
    __device__ __forceinline__ Pair shared(int t, int i, int run) const {
        return run < (int)size * kWarps ? Pair{sm->seg[t][i][run], sm->seg[t][i + 1][run]} : Pair{0.f, 0.f};
    }
    __device__ __forceinline__ unsigned shared_count(int t, int run) const {
        return run < (int)size * kWarps ? __float_as_uint(sm->seg[t][4][run]) : 0u;
    }
    // The row's sum of what its warps shared.
    __device__ Pair shared_sum(int t, int i) const { return warp_sum(shared(t, i, lane) + shared(t, i, lane + 32)); }

    // Sum over the block's threads below this one.
    template <typename V, typename S>
    __device__ V before(V x, S* scratch, V& total) {
        const V below = lanes_below(x, lane);
        __syncthreads();
        if (lane == 31) *reinterpret_cast<V*>(&scratch[warp]) = below + x;
        __syncthreads();
        V b{};
        total = V{};
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const V y = *reinterpret_cast<const V*>(&scratch[w]);
            if (w < warp) b = b + y;
            total = total + y;
        }
        return b + below;
    }
    // The nearest bins of sm->tot that are not empty before and behind `bin` (0, kBins - 1 where there is none).
    __device__ void neighbours(int bin, int& prev, int& next) {
        constexpr int kEach = kBins / kThreads;
        if (tid == 0) sm->found_prev = 0, sm->found_next = kBins - 1;
        __syncthreads();
        int p = 0, n = kBins - 1;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int b = tid * kEach + i;
            if (sm->tot[b] && b < bin) p = b;
            if (sm->tot[b] && b > bin) n = min(n, b);
        }
        p = __reduce_max_sync(0xffffffffu, p);
        n = __reduce_min_sync(0xffffffffu, n);
        if (lane == 0) {
            atomicMax(&sm->found_prev, p);
            atomicMin(&sm->found_next, n);
        }
        __syncthreads();
        prev = sm->found_prev;
        next = sm->found_next;
        __syncthreads();
    }
    // The least of the block's numbers, in every thread.
    __device__ int lowest(int x) {
        if (tid == 0) sm->found = x;
        x = __reduce_min_sync(0xffffffffu, x);
        __syncthreads();
        if (lane == 0) atomicMin(&sm->found, x);
        __syncthreads();
        x = sm->found;
        __syncthreads();
        return x;
    }
    // The bin of sm->tot that holds the k-th token (k >= 1): its number, -1 if there are fewer, and the tokens before it.
    __device__ int bin_of_rank(unsigned k, unsigned& above) {
        constexpr int kEach = kBins / kThreads;
        unsigned n[kEach], s = 0, total;
#pragma unroll
        for (int i = 0; i < kEach; ++i) s += n[i] = sm->tot[tid * kEach + i];
        unsigned c = before(s, sm->scan_u, total);
        if (tid == 0) sm->found = -1;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            if (c < k && k <= c + n[i]) {
                sm->found = tid * kEach + i;
                sm->found_count = c;
            }
            c += n[i];
        }
        __syncthreads();
        const int b = sm->found;
        above = sm->found_count;
        __syncthreads();
        return b;
    }
};

// Keys whose first bin is b or less begin at this one (bin_of falls with the key).
template <int kDrop>
__device__ __forceinline__ uint32_t lowest_key(int b, float m, float c32, uint32_t none, uint32_t top) {
    uint32_t lo = none, hi = top;  // bin(hi) <= b; the answer is in (lo, hi]
    while (hi - lo > 1) {
        const uint32_t mid = lo + (hi - lo) / 2;
        if (bin_of(of_key<kDrop>(mid), m, c32) <= b) hi = mid;
        else lo = mid;
    }
    return hi;
}

// How far keys of a range of this length are shifted so that they fall into kBins.
__device__ __forceinline__ int shift_of(uint32_t range) { return max(0, 22 - __clz(range)); }  // 32 - clz = bits; bits - 10

template <typename T>
__global__ void __launch_bounds__(kThreads, 3) sample_kernel(const SampleArgs a) {
    using R = Row<T>;
    constexpr int kPer = R::kPer, kDrop = R::kDrop;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Smem* sm = reinterpret_cast<Smem*>(smem_raw);
    uint4* held = reinterpret_cast<uint4*>(sm + 1);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    R r;
    r.sm = sm;
    r.rank = cluster_rank();
    r.size = cluster_size();
    r.tid = threadIdx.x;
    r.lane = r.tid & 31;
    r.warp = r.tid >> 5;
    r.turn = 0;
    r.list_lo = 1, r.list_hi = 0;
    const int row = blockIdx.x / r.size;
    const long long first = (long long)r.rank * a.chunk;
    r.len = (int)max(0ll, min((long long)a.chunk, a.V - first));
    r.chunk = static_cast<const T*>(a.logits) + row * a.row_stride + first;
    r.mis = (int)((reinterpret_cast<uintptr_t>(r.chunk) & 15) / sizeof(T));
    r.held = held;
    r.resident = a.resident;
    const int words = r.len > 0 ? (r.len + r.mis + kPer - 1) / kPer : 0;
    const int run = (words + kWarps - 1) / kWarps;
    r.w0 = min(words, r.warp * run);
    r.w1 = min(words, r.w0 + run);

    // ---- the row into shared memory, its largest logit
    float m = kNegInf;
    bool bad = false;
    constexpr int kAhead = 4;
    for (int w = r.w0 + r.lane; w < r.w1; w += 32 * kAhead) {
        uint4 x[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (w + 32 * j < r.w1) x[j] = r.load(w + 32 * j);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (w + 32 * j >= r.w1) break;
            if (w + 32 * j < a.resident) held[w + 32 * j] = x[j];
            float z[kPer];
            Logits<T>::floats(x[j], z);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                bad |= !(z[i] < -kNegInf);
                m = fmaxf(m, z[i]);
            }
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float t = a.temperature ? a.temperature[row] : 1.f;
    const float u = a.uniform[row];
    int k = a.top_k ? a.top_k[row] : 0;
    const float p = a.top_p ? a.top_p[row] : 1.f;
    const float min_p = a.min_p ? a.min_p[row] : 0.f;
    bad |= !(t >= 0.f) || !(u >= 0.f && u < 1.f) || p != p || min_p != min_p;
    bad = __any_sync(0xffffffffu, bad);
    cluster_sync();  // every CTA of the cluster runs: its shared memory may be written
    int s = r.share(Pair{m, 0.f}, Pair{0.f, 0.f}, bad);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (r.lane + 32 * i < (int)r.size * kWarps) {
            m = fmaxf(m, sm->seg[s][0][r.lane + 32 * i]);
            bad |= r.shared_count(s, r.lane + 32 * i) != 0;
        }
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    bad = __any_sync(0xffffffffu, bad);
    const bool writer = r.rank == 0 && r.tid == 0;
    if (bad || m == kNegInf) {  // (alike in every thread of the cluster)
        if (writer) {
            if (bad) atomicOr(a.err, kErrBadValue);
            a.out_tokens[row] = -1;
            if (a.out_logprobs) a.out_logprobs[row] = kNegInf;
        }
        return;
    }
    m += 0.f;  // (-0 is 0)
    if (k >= a.V || k < 0) k = 0;
    const uint32_t top = key_of<kDrop>(m);

    if (t == 0.f || k == 1 || p <= 0.f) {  // the first of the largest
        unsigned at = 0xFFFFFFFFu;
        for (int it = 0, n = r.steps(); it < n && at == 0xFFFFFFFFu; ++it) {
            float z[kPer];
            r.step(r.w0, r.w1, it, z);
            unsigned mine = 0xFFFFFFFFu;
#pragma unroll
            for (int i = kPer - 1; i >= 0; --i)
                if (z[i] == m) mine = (unsigned)(first + r.token(r.w0 + it * 32 + r.lane, i));
            at = __reduce_min_sync(0xffffffffu, mine);
        }
        s = r.share(Pair{0.f, 0.f}, Pair{0.f, 0.f}, at);
        if (writer) {
            for (int i = 0; i < (int)r.size * kWarps; ++i) at = min(at, r.shared_count(s, i));
            a.out_tokens[row] = (int)at;
            if (a.out_logprobs) a.out_logprobs[row] = 0.f;
        }
        return;
    }

    Weight g;
    static_cast<RowScale&>(g) = row_scale(m, t);
    {
        const float2 root = kRoots[r.lane];
        g.th = root.x;
        g.tl = root.y;
    }
    if (min_p > 0.f && r.tid == 0) {  // the least logit whose weight reaches min_p; in 64 bits, once a CTA
        const double low = (double)m + (double)t * log((double)fminf(min_p, 1.f));
        sm->cutoff = min_p >= 1.f ? m : __double2float_ru(low);
    }

    const float c32 = fmaxf(-kBinsPerOctave * g.ch, -3e38f);
    // What is kept: keys above `keep`, and the first `ties` of those equal to it.
    uint32_t keep = R::kNone;
    unsigned ties = 0;
    Pair seg_a = {0.f, 0.f};  // this warp's sum of the weights above `summed`
    uint32_t summed = 0xFFFFFFFFu;

    const bool with_p = p < 1.f;
    int pbin = 0, pbin_prev = 0, pbin_next = kBins - 1;  // the first bin in which top-p alone should end, and the bins beside it
    if (k > 0 || with_p) r.count_bins(m, c32);
    if (with_p && k == 0) {
        // this thread's bins' weight, by their middles
        constexpr int kEach = kBins / kThreads;
        unsigned n[kEach];
        float w[kEach], est = 0.f, all;
#pragma unroll
        for (int i = 0; i < kEach; ++i) n[i] = sm->tot[r.tid * kEach + i];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            w[i] = (float)n[i] * fast_exp2(-((float)(r.tid * kEach + i) + 0.5f) / kBinsPerOctave);
            est += w[i];
        }
        float b = r.before(est, sm->scan_f, all);
        pbin = min(r.lowest(first_reaching(b, w, n, p * all, r.tid * kEach, kBins)), kBins - 1);
        r.neighbours(pbin, pbin_prev, pbin_next);
    }

    // Both borders from the sorted candidates: `of` of them (0: all) stay by top-k, and of those (with_p) the ones before which the sum,
    // from `base` on, is below `limit` (known: p of the sum of all).  False: it does not end among them.
    auto among_sorted = [&](int n, int of, Pair base, bool known, Pair limit) {
        constexpr int kEach = kSort / kThreads;
        const int stay = of ? min(of, n) : n;
        int last = stay - 1;
        if (with_p) {
            Pair w[kEach], mass = {0.f, 0.f}, total;
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int j = r.tid * kEach + i;
                w[i] = weight1(g, of_key<kDrop>(j < stay ? sm->hist[j] : top));
                if (j >= stay) w[i] = {0.f, 0.f};
                mass = mass + w[i];
            }
            Pair b = base + r.before(mass, sm->scan_p, total);
            if (!known) limit = times(total, p);
            if (known && base + total < limit) return false;
            if (r.tid == 0) sm->found = 0;
            __syncthreads();
            int mine = 0;
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int j = r.tid * kEach + i;
                if (j < stay && b < limit) mine = j;
                b = b + w[i];
            }
            mine = __reduce_max_sync(0xffffffffu, mine);
            if (r.lane == 0) atomicMax(&sm->found, mine);
            __syncthreads();
            last = sm->found;
            __syncthreads();
        }
        keep = sm->hist[last];
        for (int j = r.tid; j <= last; j += kThreads)
            if (sm->hist[j] == keep && (j == 0 || sm->hist[j - 1] != keep)) sm->found = j;
        __syncthreads();
        ties = (unsigned)(last - sm->found) + 1u;
        __syncthreads();
        return true;
    };
    bool done = false;

    // ---- top-k
    if (k > 0) {
        unsigned above;
        const int b = r.bin_of_rank((unsigned)k, above);
        if (b >= 0) {  // (else fewer tokens than k are not -inf)
            uint32_t khi = b == 0 ? top : lowest_key<kDrop>(b - 1, m, c32, R::kNone, top) - 1;
            uint32_t klo = lowest_key<kDrop>(b, m, c32, R::kNone, top);
            const unsigned candidates = above + sm->tot[b];
            r.make_list(klo, 0xFFFFFFFFu);  // all that can stay
            int n;
            if (candidates <= kSort && r.sort_lists(n)) done = among_sorted(n, k, Pair{0.f, 0.f}, false, Pair{0.f, 0.f});
            for (int round = 0; !done && klo < khi && round < 8; ++round) {  // (four rounds take 32 bits to one value)
                const int shift = shift_of(khi - klo);
                r.count_keys(klo, khi, shift);
                unsigned more;
                const int c = r.bin_of_rank((unsigned)k - above, more);
                if (c < 0) break;
                above += more;
                khi -= (uint32_t)c << shift;
                klo = max(klo, khi - min(khi, (1u << shift) - 1u));
            }
            if (!done) {
                keep = khi;
                ties = (unsigned)k - above;
            }
        }
    }

    // ---- top-p
    if (with_p && !done) {
        const uint32_t bottom = keep;  // what top-k keeps
        const unsigned bottom_ties = ties;
        // keys at which top-p may end: from `least`, which is `bottom` itself if top-k keeps some of it, to `most`; both follow what
        // the exact sums say
        uint32_t least = bottom + (bottom_ties ? 0u : 1u), most = top;
        uint32_t khi = pbin_prev == 0 ? top : lowest_key<kDrop>(pbin_prev - 1, m, c32, R::kNone, top) - 1;
        uint32_t klo = pbin_next == kBins - 1 ? least : lowest_key<kDrop>(pbin_next, m, c32, R::kNone, top);
        klo = max(klo, least);
        khi = max(khi, klo);
        Pair target = {0.f, 0.f};
        bool known = false;
        for (int round = 0; round < 200; ++round) {  // (a handful; at worst each halves what is left of 2^32 keys)
            // the weights above the window (at first with the sum of all), and the counts in it
            const int shift = shift_of(khi - klo);
            Pair rest = {0.f, 0.f};
            unsigned none;
            if (!known) {
                r.sum_apart(g, bottom, khi, klo, shift, seg_a, rest);
            } else {
                seg_a = seg_a + r.sum(g, khi, summed, none);
                r.count_keys(klo, khi, shift);
            }
            summed = khi;
            s = r.share(seg_a, rest, 0u);
            const Pair above = r.shared_sum(s, 0);
            if (!known) {
                Pair all = above + r.shared_sum(s, 2);
                if (bottom_ties) all = all + times(weight1(g, of_key<kDrop>(bottom)), bottom_ties);
                target = times(all, p);
                known = true;
            }
            if (!(above < target)) {  // it ends above the window
                if (khi >= most) {    // ... which a rounding of the sums says only, at a key's very border
                    keep = khi;
                    ties = 0;
                    break;
                }
                least = klo = khi + 1;
                khi = most;
                seg_a = {0.f, 0.f};
                summed = 0xFFFFFFFFu;
                continue;
            }
            most = khi;
            constexpr int kEach = kBins / kThreads;
            if (shift > 0 && bottom_ties == 0) {  // few enough to be sorted?
                unsigned c = 0, all;
#pragma unroll
                for (int i = 0; i < kEach; ++i) c += sm->tot[r.tid * kEach + i];
                r.before(c, sm->scan_u, all);
                if (all <= kSort && all > 0) {
                    r.make_list(klo, khi);
                    int n;
                    if (r.sort_lists(n) && among_sorted(n, 0, above, true, target)) break;
                }
            }
            Pair w[kEach], mass = {0.f, 0.f}, total;
            unsigned n[kEach];
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const uint32_t bin = r.tid * kEach + i;
                const uint32_t hi = khi - min(khi - klo, bin << shift);  // (bins behind the window are empty)
                const uint32_t lo = max(klo, hi - min(hi, (1u << shift) - 1u));
                n[i] = sm->tot[bin];
                if (bottom_ties && shift == 0 && hi == bottom) n[i] = min(n[i], bottom_ties);
                w[i] = times(weight1(g, of_key<kDrop>(lo + (hi - lo) / 2)), n[i]);
                mass = mass + w[i];
            }
            Pair b = above + r.before(mass, sm->scan_p, total);
            const int mine = first_reaching(b, w, n, target, r.tid * kEach, kBins);
            int bin = r.lowest(mine);
            if (bin == kBins) {
                bin = -1;
            } else if (bin == mine) {  // (one thread's: bins are dealt apart)
                sm->found_mass = make_float2(b.h, b.l);
#pragma unroll
                for (int i = 0; i < kEach; ++i)
                    if (bin == r.tid * kEach + i) sm->found_count = n[i];
            }
            __syncthreads();
            const Pair b0 = {sm->found_mass.x, sm->found_mass.y};
            const unsigned here = sm->found_count;
            __syncthreads();
            if (bin < 0 && shift == 0) {  // it ends below the window
                if (klo <= least) {       // ... which a rounding of the sums says only: all stays that top-k keeps
                    keep = bottom;
                    ties = bottom_ties;
                    break;
                }
                most = khi = klo - 1;
                klo = least;
                continue;
            }
            if (shift == 0) {
                // of the ties, those before which the sum is still below the target
                keep = khi - (uint32_t)bin;
                const Pair wk = weight1(g, of_key<kDrop>(keep));
                if (r.tid == 0) {
                    const double want = ceil((value(target) - value(b0)) / value(wk));
                    sm->found_count = want < 1.0 ? 1u : want > (double)here ? here : (unsigned)want;
                }
                __syncthreads();
                ties = sm->found_count;
                __syncthreads();
                break;
            }
            // narrower, by the middles' weights, with a bin that is not empty on each side; where that is not much narrower, or they
            // say nothing, the next sums decide for one half
            const uint32_t half = klo + (khi - klo) / 2;
            if (bin >= 0) {
                int prev, next;
                r.neighbours(bin, prev, next);
                const uint32_t high = khi - ((uint32_t)prev << shift);
                const unsigned long long down = ((unsigned long long)(next + 1) << shift) - 1u;
                const uint32_t low = khi - klo > down ? khi - (uint32_t)down : klo;
                if (high - low <= (khi - klo) / 2) {
                    klo = low;
                    khi = high;
                    continue;
                }
            }
            khi = half;
        }
    }

    // ---- min-p: weights of at least min_p
    if (min_p > 0.f) {
        __syncthreads();
        const uint32_t full = key_of<0>(sm->cutoff);
        const uint32_t low = kDrop == 0 || !(full >> 31) ? full >> kDrop : (full >> kDrop) + ((full & ((1u << kDrop) - 1u)) ? 1u : 0u);
        if (low > keep) {
            keep = min(low, top) - 1;
            ties = 0;
        }
    }

    // ---- the sums by run, and the run that holds the token
    if (keep > summed) {
        seg_a = {0.f, 0.f};
        summed = 0xFFFFFFFFu;
    }
    {
        unsigned n;
        seg_a = seg_a + r.sum(g, keep, summed, n);
        s = r.share(seg_a, Pair{0.f, 0.f}, n);
    }
    const Pair wk = weight1(g, of_key<kDrop>(ties ? keep : top));
    if (!(wk.h > 0.f)) ties = 0;  // (what has no weight is not picked)
    // kept weight up to a place: those above `keep` before it, and as many of its ties as are kept
    auto kept = [&](Pair sum, unsigned n) { return ties ? sum + times(wk, min(n, ties)) : sum; };
    Pair at_a;  // before the place looked for
    unsigned at_t;
    Pair Z, target;
    int owner;
    {
        const Pair s0 = r.shared(s, 0, 2 * r.lane), s1 = r.shared(s, 0, 2 * r.lane + 1);
        const unsigned n0 = r.shared_count(s, 2 * r.lane), n1 = r.shared_count(s, 2 * r.lane + 1);
        const Pair b0 = lanes_below(s0 + s1, r.lane), b1 = b0 + s0, b2 = b1 + s1;
        const unsigned c0 = lanes_below(n0 + n1, r.lane), c1 = c0 + n0, c2 = c1 + n1;
        const Pair k0 = kept(b0, c0), k1 = kept(b1, c1), k2 = kept(b2, c2);
        Z = Pair{__shfl_sync(0xffffffffu, k2.h, 31), __shfl_sync(0xffffffffu, k2.l, 31)};
        target = times(Z, u);
        // the last run whose kept weights begin at or before the target and are not nothing
        const bool in0 = k0 < k1 && !(target < k0), in1 = k1 < k2 && !(target < k1);
        const unsigned may = __ballot_sync(0xffffffffu, in0 || in1);
        const int who = may ? 31 - __clz(may) : 0;
        owner = __shfl_sync(0xffffffffu, 2 * r.lane + (in1 ? 1 : 0), who);
        at_a = Pair{__shfl_sync(0xffffffffu, in1 ? b1.h : b0.h, who), __shfl_sync(0xffffffffu, in1 ? b1.l : b0.l, who)};
        at_t = __shfl_sync(0xffffffffu, in1 ? c1 : c0, who);
    }
    if (owner / kWarps != (int)r.rank) return;

    // ---- the last step of that run that has some kept weight and begins at or before the target, every warp of its CTA summing some
    // (Whether a step, a lane or a token has weight is asked of its own sum and count, not of the sums before and behind it: these may
    // round to the same, and a run be found whose steps all do.  The first that has weight begins where the run does, so there is one.)
    const int ow = owner % kWarps;
    const int a0 = min(words, ow * run), a1 = min(words, a0 + run);
    const bool list = r.listed(ties ? keep : keep + 1u, 0xFFFFFFFFu, ow);
    const int n_steps = list ? r.list_steps(ow) : (a1 - a0 + 31) / 32;
    auto lane_sums = [&](int it, float (&z)[kPer], uint32_t (&key)[kPer], Pair& sa, unsigned& st) {
        if (list) r.list_step(ow, it, z);
        else r.step(a0, a1, it, z);
        float2 hi = both(0.f), lo = both(0.f);
        st = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            key[i] = key_of<kDrop>(z[i]);
            st += key[i] == keep;
        }
        const float zkeep = bound_of<kDrop>(keep);
        R::add_weights(g, z, [&](float x) { return x > zkeep; }, hi, lo);
        sa = R::joined(hi, lo);
    };
    int best = -1;
    Pair best_a = at_a;
    unsigned best_t = at_t;
    float z[kPer];
    uint32_t key[kPer];
    Pair sa;
    unsigned st;
    for (int base = 0; base < n_steps; base += kBatch) {
        __syncthreads();
        for (int it = base + r.warp; it < min(n_steps, base + kBatch); it += kWarps) {
            lane_sums(it, z, key, sa, st);
            sa = warp_sum(sa);
            st = __reduce_add_sync(0xffffffffu, st);
            if (r.lane == 0) {
                sm->step_a[it - base] = make_float2(sa.h, sa.l);
                sm->step_t[it - base] = st;
            }
        }
        __syncthreads();
        if (r.warp == 0) {
            for (int it = base; it < min(n_steps, base + kBatch); ++it) {
                const Pair here = {sm->step_a[it - base].x, sm->step_a[it - base].y};
                const unsigned here_t = sm->step_t[it - base];
                if ((here.h > 0.f || (here_t && at_t < ties)) && !(target < kept(at_a, at_t))) {
                    best = it;
                    best_a = at_a;
                    best_t = at_t;
                }
                at_a = at_a + here;
                at_t += here_t;
            }
        }
    }
    if (r.warp != 0) return;

    // ---- the last lane, and in it the last token, whose kept weight begins at or before the target and is not nothing
    const Pair wm = weight1(g, m);  // (all lanes)
    lane_sums(best, z, key, sa, st);
    Pair ca = best_a + lanes_below(sa, r.lane);
    unsigned ct = best_t + lanes_below(st, r.lane);
    const unsigned may = __ballot_sync(0xffffffffu, (sa.h > 0.f || (st && ct < ties)) && !(target < kept(ca, ct)));
    const int who = 31 - __clz(may);
    int token = -1;
    float picked = m;
#pragma unroll
    for (int i = 0; i < kPer; i += 2) {
        float2 vl;
        const float2 v = weights2(g, make_float2(z[i], z[i + 1]), vl);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const bool takes = (key[i + j] > keep && (j ? v.y : v.x) > 0.f) || (key[i + j] == keep && ct < ties);
            if (takes && (token < 0 || !(target < kept(ca, ct)))) {
                token = (int)first + (list ? sm->list_at[ow][(best * 32 + r.lane) * kPer + i + j] : r.token(a0 + best * 32 + r.lane, i + j));
                picked = z[i + j];
            }
            if (key[i + j] > keep) ca = ca + (j ? Pair{v.y, vl.y} : Pair{v.x, vl.x});
            ct += key[i + j] == keep;
        }
    }
    if (r.lane == who) {
        a.out_tokens[row] = token;
        if (a.out_logprobs) a.out_logprobs[row] = (float)(((double)picked - (double)m) / (double)t - log(value(Z) / value(wm)));
    }
}

template <typename T>
cudaError_t launch(SampleArgs a, cudaStream_t stream) {
    constexpr int kPer = Logits<T>::kPer;
    int dev = 0, sms = 0, most = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    if (e != cudaSuccess) return e;
    static thread_local bool done[64] = {};
    if ((e = allow_all_smem(reinterpret_cast<const void*>(sample_kernel<T>), dev, done)) != cudaSuccess) return e;
    // CTAs a row: as many as it takes to keep a chunk within what lets three CTAs share an SM (52 KB beside 22 KB of Smem; the registers
    // allow three, which hide each other's waits), more while the rows leave SMs without work and a chunk has a few thousand tokens left.
    // Rows that eight such chunks cannot hold have larger ones, and fewer CTAs an SM.
    const size_t room = 52 * 1024;
    int size = 1;
    while (size < kMaxCluster && (size_t)a.V * sizeof(T) > room * size) size *= 2;
    while (size < kMaxCluster && (long long)a.N * size * 2 <= sms && a.V / (size * 2) >= 2048) size *= 2;
    a.chunk = ((a.V + size - 1) / size + 7) & ~7;
    const int words = a.chunk / kPer + 1;  // (a chunk that does not begin at a 16-byte boundary has one more)
    const int fit = (int)(((size_t)most - sizeof(Smem) - 64) / 16);
    a.resident = words < fit ? words : fit;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)size;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)a.N * size));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Smem) + (size_t)a.resident * 16;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, sample_kernel<T>, a);
}

}  // namespace

cudaError_t sample_launch(const SampleArgs& a, cudaStream_t stream) {
    if (a.N == 0) return cudaSuccess;
    if (a.dtype == 0) return launch<float>(a, stream);
    if (a.dtype == 1) return launch<__nv_bfloat16>(a, stream);
    return launch<__half>(a, stream);
}

}  // namespace sinkattn
