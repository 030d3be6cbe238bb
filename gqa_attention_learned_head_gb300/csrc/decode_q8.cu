// decode_q8.cu -- paged split-KV decode over a cache held in 8 bits, with a per-head learned sink.
//
// Source of the method: "GPT-OSS on day 0" (Perplexity), section "Kernels for GPT-OSS / Sink Attention" (attention parallel over heads
// and along the KV length, online softmax, the sink in one block only); the posts hold their cache in 16 bits, the 8-bit form is
// this library's.  Keys and values are codes (e4m3) with a power of two 2^ek, 2^ev for each page of 16 tokens and KV head:
//     s_j = scale 2^ek(j) <q, ck_j>,   out = sum_j e^(s_j - M) 2^ev(j) cv_j / Z,   Z = e^(sink - M) + sum_j e^(s_j - M).
//
// The work split, the deal of pages to warps, the barrier-free piece ends and the merge launched behind are those of decode.cu.  What
// 8 bits change:
//  * Half the bytes in flight a page, so twice the ring stages: a page's K and V are contiguous 1 KiB slices, fetched by two bulk
//    copies into one of kStages stages of each warp.  No tensor map: the fragment orders below need no swizzle.
//  * mma.m16n8k16 takes f16 operands, into which codes convert exactly and two at a time.  The query row is multiplied by the power
//    of two that puts its largest value into [2^14, 2^15): bf16's 8 bits are exact in f16 down to 2^-31 of that.
//  * K needs no ldmatrix: the sum over the head dimension may run in any order, so a lane's four k-columns of each product are four
//    neighbouring dimensions, and it reads its 16 dimensions of two tokens with two 16-byte loads.
//  * V^T needs pairs of tokens in one register: four tokens' 8 dimensions are read with 8-byte loads and interleaved with byte
//    permutes before they are converted.  Which token stands in which row of the score tile is free too: token_of() puts the pairs of
//    K loads on different banks, and half of the V loads.
//  * The value scale goes into the weights where it is within 2^2 of the scale 2^eo that a warp's accumulators have:
//    w_j = 2^(x_j - R + ev(j) - eo), x the scores in base 2, R a running bound of x (raised, and O scaled down, only when a page exceeds
//    it by more than kSlack).  They are held in f16, whose 11 bits round less than the bf16 output; kLift keeps w above f16's
//    subnormals down to 2^-21 of the row's largest, and off by at most 2^-32 of it below.  A page further off gives the accumulators its
//    own scale first (a power of two: exact).  Where its scale is more than 2^kSpread above another's, what its weights lose below
//    2^-21 could outweigh the others: it takes them relative to its own largest, and its products are joined in 32 bits.  So one
//    large value neither hides the other pages' dimensions nor is lost at a low score.  The sum of the weights is
//    kept relative to R, without scales.  The sink joins when a piece ends, by its logarithm.
//
//  * Two pages are taken together: their bounds are compared before they are reduced over the lanes (only where one exceeds R does
//    any shuffle run), and one turn of the loop waits, refills and branches for both.
//
// 2 x (64 + 1/16) bytes a token and KV head, 1/16 of it scales.  Measured (GB300): 4 x 131072 tokens 101 us, 5.3 TB/s = 79% of the
// copy rate; 32 requests of 512 to 4096 tokens 31 us; one of 128 tokens 5.4.  What bounds the long case is no longer HBM alone: with half the
// bytes a page, the same instructions a page take half of all issue slots, most of the rest waiting on the instruction before
// (four warps a scheduler at 128 registers).  One page at a time: 118 us; two, with branches
// for short and missing pages among their instructions: 105.  Products of codes with codes (the query as the sum
// of two codes), which need no conversion of K: 120 us against 105, the fp8 form of mma.sync being no faster and K's conversions no longer
// hidden.  Rings of 5 or 6 stages: 132, 121 us (fewer CTAs an SM); shares of at least 64 pages instead of 32: no change.  Weights with
// all of the value scale in them, relative to a bound of x + ev, took 98 us and lost pages 2^25 and more below the largest scale.
#include <type_traits>

#include "args_merge.h"
#include "args_q8.h"
#include "ptx.cuh"
#include "q8.cuh"
#include "smem_limit.h"
#include "split_kv.cuh"

#ifndef SINKATTN_DECODE_Q8_STAGES
#define SINKATTN_DECODE_Q8_STAGES 4
#endif
#ifndef SINKATTN_DECODE_Q8_MIN_PAGES
#define SINKATTN_DECODE_Q8_MIN_PAGES 32
#endif

namespace sinkattn {
namespace {

constexpr int kWarps = 4;
constexpr int kStages = SINKATTN_DECODE_Q8_STAGES;
constexpr int kSliceBytes = kPageSize * kHeadDim;  // 1024: one (page, KV head) of K or V
constexpr int kStageBytes = 2 * kSliceBytes;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLift = 9.f;  // weights are 2^kLift times their size, at most 2^(kLift + kSlack + kWindow) = 2^15 < 65504
constexpr float kSlack = 4.f;
constexpr int kWindow = 2;    // value exponents this near to the accumulators' go into the weights
constexpr int kSpread = 6;    // pages of value exponents further than this above another's take weights relative to their own largest

// The token of a page that row r of its score tile holds (r + 8: the same + 8).
__device__ __forceinline__ int token_of(int r) { return (int)(0x65742130u >> (4 * r)) & 7; }

// Shared memory: ring | mbarriers | stage words | combine slots | slot words | scan | prefix[B+1].
template <int NT>
struct SmemLayout {
    static constexpr int kHeads = 8 * NT;
    static constexpr size_t ring = size_t(kWarps) * kStages * kStageBytes;
    static constexpr size_t bars = ring;
    static constexpr size_t meta = bars + size_t(kWarps) * kStages * 8;
    static constexpr size_t cmb_o = (meta + size_t(kWarps) * kStages * 4 + 15) & ~size_t(15);  // [2][warps][heads][64] f32
    static constexpr size_t cmb_md = cmb_o + 2 * size_t(kWarps) * kHeads * kHeadDim * 4;       // [2][warps][heads] R, d
    static constexpr size_t slot = cmb_md + 2 * size_t(kWarps) * kHeads * 8;                   // [2] arrivals, [2] generation
    static constexpr size_t scan = slot + 4 * 4;                                               // [kWarps] scan scratch
    static constexpr size_t least = scan + kWarps * 4;                                         // [kWarps] least value exponents
    static constexpr size_t prefix = least + kWarps * 4;
    static constexpr size_t fixed = prefix + 128 /* alignment slack */;
};

__device__ __forceinline__ void bulk_load(void* dst, const uint8_t* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}
// D[16x8] += A[16x16] * B[16x8], f16 inputs, fp32 accumulate.
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t min_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// log2(2^a + 2^b), either may be infinite.
__device__ __forceinline__ float log2_sum(float a, float b) {
    const float m = fmaxf(a, b);
    return fabsf(m) == -kNegInf ? m : m + log2f(exp2f(a - m) + exp2f(b - m));
}

// A piece as the decode processes it (see decode.cu): `rot` is the warp whose turn it is at the piece's first page.
struct Piece : SegPiece {
    int rot;
    __device__ bool split() const { return len() >= kWarps; }
    __device__ int offset(int w) const { return (w - rot + kWarps) % kWarps; }
    __device__ int count(int w) const {
        if (split()) {
            const int o = offset(w);
            return len() > o ? (len() - o + kWarps - 1) / kWarps : 0;
        }
        return rot == w ? len() : 0;
    }
    __device__ int page(int w, int t) const { return page0() + (split() ? offset(w) + t * kWarps : t); }
    __device__ void first(const int* prefix, int B, int Hkv, long long x0, long long x1) {
        piece_first(*this, prefix, B, Hkv, x0, x1);
        rot = 0;
    }
    __device__ void next(const int* prefix, int B, int Hkv, long long x1) {
        rot = (rot + len()) % kWarps;
        piece_next(*this, prefix, B, Hkv, x1);
    }
};

// Bounded spin until a shared-memory word reaches `want`; false on give-up.
__device__ __forceinline__ bool wait_word(const int* w, int want) {
    for (uint32_t i = 0; i < kMaxPolls; ++i)
        if (*reinterpret_cast<const volatile int*>(w) == want) return true;
    return false;
}

template <int NT>  // NT = ceil(G / 8) groups of 8 query heads
__global__ void __launch_bounds__(kWarps * 32, NT == 1 ? 4 : 3) decode_q8_kernel(const DecodeQ8Args a) {
    using L = SmemLayout<NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::bars);
    uint32_t* meta = reinterpret_cast<uint32_t*>(sm + L::meta);
    float* cmb_o = reinterpret_cast<float*>(sm + L::cmb_o);
    float* cmb_md = reinterpret_cast<float*>(sm + L::cmb_md);
    int* slot_arr = reinterpret_cast<int*>(sm + L::slot);  // [2] warps counted in for the slot's piece
    int* slot_gen = slot_arr + 2;                          // [2] pieces the slot has combined
    int* scan = reinterpret_cast<int*>(sm + L::scan);
    int* prefix = reinterpret_cast<int*>(sm + L::prefix);  // [B + 1] exclusive prefix of pages per request

    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int B = a.B, Hkv = a.Hkv, G = a.G, cap = a.max_pages * kPageSize;
    const long long cta = blockIdx.x;

    // ---- 1. pages per request -> exclusive prefix sum (every CTA, in shared memory)
    int running = 0;
    for (int base = 0; base < B; base += kWarps * 32) {
        int b = base + tid, n = 0;
        if (b < B) {
            int Lb = a.kv_lens[b];
            if ((Lb < 0 || Lb > cap) && blockIdx.x == 0) atomicOr(a.err, kErrBadLength);
            n = (clamp_len(Lb, cap) + kPageSize - 1) / kPageSize;
        }
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) scan[warp] = incl;
        __syncthreads();
        int woff = 0, tot = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            int v = scan[w];
            woff += (w < warp) ? v : 0;
            tot += v;
        }
        if (b < B) prefix[b] = running + woff + incl - n;
        running += tot;
        __syncthreads();
    }
    if (tid == 0) {
        prefix[B] = running;
        slot_arr[0] = slot_arr[1] = 0;
        slot_gen[0] = slot_gen[1] = 0;
    }
    __syncthreads();

    // ---- 2. requests with no cached token: all mass on the sink (out = 0, lse = sink)
    {
        const long long rows = (long long)B * a.Hq;
        for (long long r = (long long)blockIdx.x * blockDim.x + tid; r < rows; r += (long long)gridDim.x * blockDim.x) {
            const int b = (int)(r / a.Hq);
            if (prefix[b + 1] != prefix[b]) continue;
            uint4* dst = reinterpret_cast<uint4*>(a.out + r * kHeadDim);
#pragma unroll
            for (int c = 0; c < 8; ++c) dst[c] = make_uint4(0, 0, 0, 0);
            if (a.lse) a.lse[r] = __ldg(&a.sinks[r - (long long)b * a.Hq]);
        }
    }

    const long long U = (long long)running * Hkv;
    const long long C = U > 0 ? effective_shares(a.workers, a.fixed_workers, a.min_pages_per_worker, U) : 0;
    if (cta >= C) {
        if (tid == 0 && a.merge_list) a.merge_list[cta] = make_int2(-1, 0);
        return;
    }
    const long long x0 = cta * U / C, x1 = (cta + 1) * U / C;

    uint8_t* my_ring = sm + warp * kStages * kStageBytes;
    uint64_t* my_bars = bars + warp * kStages;
    uint32_t* my_meta = meta + warp * kStages;  // a stage's scale bytes, keys' | values' << 16; 0: its page id was out of range
    if (lane == 0) {
        for (int s = 0; s < kStages; ++s) mbar_init(&my_bars[s], 1);
        fence_mbar_init();
        fence_proxy_async_smem();
    }
    __syncwarp();

    // ---- 3. producer: walks this warp's units piece by piece, two pages at a time; the lanes resolve 32 page ids, and their scales,
    // at a time, and four of them copy: K and V of the first page, K and V of the second
    Piece pp;
    pp.first(prefix, B, Hkv, x0, x1);
    int pt = 0, pcnt = pp.count(warp), win_slice = -1, issued = 0;
    uint32_t win_scales = 0;
    auto issue = [&]() -> bool {  // warp-uniform
        while (pt >= pcnt) {
            pp.next(prefix, B, Hkv, x1);
            if (pp.ps >= x1) return false;
            pt = 0;
            pcnt = pp.count(warp);
        }
        if ((pt & 31) == 0) {
            win_slice = -1;
            win_scales = 0;
            if (pt + lane < pcnt) {
                const int pid = __ldg(&a.page_table[(long long)pp.b * a.max_pages + pp.page(warp, pt + lane)]);
                if (pid >= 0 && pid < a.num_pages) {
                    win_slice = pid * Hkv + pp.g;
                    win_scales = __ldg(reinterpret_cast<const unsigned short*>(a.kv_scales) + win_slice);
                }
            }
        }
        const int which = lane >> 1;  // 0, 1: the pages
        const int from = ((pt & 31) + which) & 31, n = min(2, pcnt - pt), s = (issued + which) % kStages;
        const int slice = __shfl_sync(0xffffffffu, win_slice, from);
        // the copies go out before the scales have come: their bytes are counted whenever they land, and the phase waits for the arrival
        if (which < n && slice >= 0)
            bulk_load(my_ring + s * kStageBytes + (lane & 1) * kSliceBytes,
                      ((lane & 1) ? a.v_pages : a.k_pages) + (long long)slice * kSliceBytes, kSliceBytes, &my_bars[s]);
        const uint32_t sc = __byte_perm(__shfl_sync(0xffffffffu, win_scales, from), 0, 0x4140);
        const uint32_t word = min_u16x2(max_u16x2(sc, 0x10001u * (kScaleExpMin + kScaleBias)), 0x10001u * (kScaleExpMax + kScaleBias));
        if (which < n && !(lane & 1)) {
            my_meta[s] = slice < 0 ? 0u : word;
            if (slice >= 0) {
                if (word != sc) atomicOr(a.err, kErrBadValue);
                mbar_arrive_expect_tx(&my_bars[s], kStageBytes);
            } else {
                atomicOr(a.err, kErrBadPage);
                mbar_arrive(&my_bars[s]);
            }
        }
        pt += n;
        issued += n;
        return true;
    };
    bool more = true;
    for (int j = 0; j < kStages / 2 && more; ++j) more = issue();

    // ---- 4. consumer: piece by piece
    const int gq = lane >> 2, tq = lane & 3;  // mma fragment coordinates
    const int tok0 = token_of(gq);            // rows gq, gq + 8 of the score tile: tokens tok0, tok0 + 8
    const int vt0 = token_of(2 * tq), vt1 = token_of(2 * tq + 1);
    float O[4][NT][4];        // [dims 8 gq + 2 mt, + 1][heads 2 tq, 2 tq + 1], times 2^(kLift - R - eo)
    int eo = kScaleBias;      // the value exponent of O, as a scale's byte
    volatile int* const least = reinterpret_cast<int*>(sm + L::least) + warp;  // (at most) the least one of the piece's pages so far
    float R[NT][2], d[NT][2];
    int consumed = 0;
    bool failed = false;  // a wait gave up: skip all further work, keep the barriers
    int nsplit = 0;       // dealt pieces met so far (they take the combine slots in turn)
    int head_seg = -1;    // segment whose page 0 this share holds without completing it

    // Per-piece inputs, fetched one piece ahead: this lane's 16 dimensions of head gq of each group, as they are in memory.
    struct PieceIn {
        uint4 q[NT][2];
        int kv_len;
    };
    auto fetch = [&](const Piece& p, PieceIn& in) {
        in.kv_len = clamp_len(__ldg(&a.kv_lens[p.b]), cap);
        const __nv_bfloat16* qb = a.q + ((long long)p.b * a.Hq + (long long)p.g * G) * kHeadDim;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int hl = nt * 8 + gq;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                in.q[nt][i] = hl < G ? __ldg(reinterpret_cast<const uint4*>(qb + hl * kHeadDim + 16 * tq) + i)
                                     : make_uint4(0, 0, 0, 0);
        }
    };
    PieceIn cur, nxt;
    Piece cp;
    cp.first(prefix, B, Hkv, x0, x1);
    fetch(cp, cur);

    while (cp.ps < x1) {
        Piece np = cp;
        np.next(prefix, B, Hkv, x1);
        if (np.ps < x1) fetch(np, nxt);  // in flight while this piece is processed

        const int cnt = cp.count(warp);
        const bool first = cp.page0() == 0;  // this piece holds the segment's page 0, and with it the sink
        const int seg = cp.b * Hkv + cp.g;
        const bool whole = first && (cp.pe == cp.seg_start + cp.n);
        if (first && !whole) head_seg = seg;

        // the query rows in f16, each times a power of two; mul: what takes a row's products to base-2 scores
        uint32_t qf[NT][4][2];
        float mul[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const uint32_t w[8] = {cur.q[nt][0].x, cur.q[nt][0].y, cur.q[nt][0].z, cur.q[nt][0].w,
                                   cur.q[nt][1].x, cur.q[nt][1].y, cur.q[nt][1].z, cur.q[nt][1].w};
            uint32_t mx = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) mx = max_u16x2(mx, w[i] & 0x7FFF7FFFu);
            mx = max(mx & 0xFFFFu, mx >> 16);
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const int ex = (int)(mx >> 7);  // the row's largest exponent field; 255: an infinity or NaN, passed on as it is
            const int up = ex == 255 ? 0 : min(14 + 127 - ex, 120);
            const float f = q8::power(up);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                qf[nt][i >> 1][i & 1] = pack_f16(__uint_as_float(w[i] << 16) * f, __uint_as_float(w[i] & 0xFFFF0000u) * f);
#pragma unroll
            for (int e = 0; e < 2; ++e)
                mul[nt][e] = a.scale_log2 * q8::power(-__shfl_sync(0xffffffffu, up, (2 * tq + e) * 4));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                R[nt][e] = kNegInf;
                d[nt][e] = 0.f;
            }
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) O[mt][nt][e] = 0.f;
        }

        for (int t = 0; t < cnt && !failed; t += 2) {
            const bool two = t + 1 < cnt;
            const int s0 = consumed % kStages, s1 = (consumed + 1) % kStages;
            bool landed = mbar_wait(&my_bars[s0], (consumed / kStages) & 1);
            if (two) landed = landed && mbar_wait(&my_bars[s1], ((consumed + 1) / kStages) & 1);
            if (!__all_sync(0xffffffffu, landed)) {
                failed = true;
                if (lane == 0) atomicOr(a.err, kErrTimeout);
                break;
            }
            const uint32_t word[2] = {my_meta[s0], two ? my_meta[s1] : 0u};
            uint8_t* const st[2] = {my_ring + s0 * kStageBytes, my_ring + s1 * kStageBytes};
            if (t == 0) {
                eo = word[0] ? (int)(word[0] >> 16) : kScaleBias;
                *least = eo - kWindow;
            }
            const int up[2] = {(int)(word[0] >> 16) - eo, (int)(word[1] >> 16) - eo};
            const bool calm = (unsigned)(up[0] + kWindow) <= 2u * kWindow && (unsigned)(up[1] + kWindow) <= 2u * kWindow;
            auto valid_of = [&](int j) { return word[j] == 0 ? 0 : min(kPageSize, cur.kv_len - cp.page(warp, t + j) * kPageSize); };
            // (two whole pages of like value scales, the usual case, without a branch, so that the instructions of both interleave)
            auto pages = [&](auto full) {
                constexpr bool kFull = decltype(full)::value;
                float x[2][NT][4], top[NT][2];
    #pragma unroll
                for (int nt = 0; nt < NT; ++nt) top[nt][0] = top[nt][1] = kNegInf;
    #pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (!kFull && j == 1 && !two) {
    #pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
    #pragma unroll
                            for (int e = 0; e < 4; ++e) x[1][nt][e] = kNegInf;
                        break;
                    }
                    const int valid = kFull ? kPageSize : valid_of(j);
                    if (valid < kPageSize) {
                        // Rows past the cache end (or a skipped page) may hold anything; zero the value rows so that
                        // 0-weight * garbage cannot produce NaN.
                        uint4* vz = reinterpret_cast<uint4*>(st[j] + kSliceBytes);
                        for (int c = valid * 4 + lane; c < kPageSize * 4; c += 32) vz[c] = make_uint4(0, 0, 0, 0);
                        __syncwarp();
                    }
                    // S^T = K Q^T : 16 tokens x 8 heads per group; product kk takes dimensions 16 tq + 4 kk .. + 3
                    const uint4 k0 = *reinterpret_cast<const uint4*>(st[j] + tok0 * kHeadDim + 16 * tq);
                    const uint4 k1 = *reinterpret_cast<const uint4*>(st[j] + (tok0 + 8) * kHeadDim + 16 * tq);
                    const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
                    float acc[NT][4];
    #pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
    #pragma unroll
                        for (int e = 0; e < 4; ++e) acc[nt][e] = 0.f;
    #pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const uint32_t af[4] = {q8::f16x2_of(w0[kk]), q8::f16x2_of(w1[kk]), q8::f16x2_of_high(w0[kk]),
                                                q8::f16x2_of_high(w1[kk])};
    #pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma_f16_16816(acc[nt], af, qf[nt][kk][0], qf[nt][kk][1]);
                    }
                    // base-2 scores; this thread holds tokens tok0, tok0 + 8 and heads 2 tq, 2 tq + 1
                    const float kf = __uint_as_float(word[j] << 23);
    #pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        // (kf first: the product of the two factors may leave f32's range where the score does not)
    #pragma unroll
                        for (int e = 0; e < 4; ++e) x[j][nt][e] = acc[nt][e] * kf * mul[nt][e & 1];
                        if (valid < kPageSize) {
    #pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (tok0 + (e >= 2 ? 8 : 0) >= valid) x[j][nt][e] = kNegInf;
                        }
    #pragma unroll
                        for (int e = 0; e < 2; ++e) top[nt][e] = fmaxf(top[nt][e], fmaxf(x[j][nt][e], x[j][nt][2 + e]));
                    }
                }

                // online softmax (base 2) over the two pages
                bool over = false;
    #pragma unroll
                for (int nt = 0; nt < NT; ++nt)
    #pragma unroll
                    for (int e = 0; e < 2; ++e) over |= top[nt][e] > R[nt][e] + kSlack;
                if (__any_sync(0xffffffffu, over)) {  // a head's bound has to rise, to the largest of its tokens
    #pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float al[2];
    #pragma unroll
                        for (int e = 0; e < 2; ++e) {
    #pragma unroll
                            for (int o = 4; o < 32; o <<= 1) top[nt][e] = fmaxf(top[nt][e], __shfl_xor_sync(0xffffffffu, top[nt][e], o));
                            const bool up = top[nt][e] > R[nt][e] + kSlack;
                            al[e] = up ? fast_exp2(R[nt][e] - top[nt][e]) : 1.f;
                            R[nt][e] = up ? top[nt][e] : R[nt][e];
                            d[nt][e] *= al[e];
                        }
    #pragma unroll
                        for (int mt = 0; mt < 4; ++mt)
    #pragma unroll
                            for (int e = 0; e < 4; ++e) O[mt][nt][e] *= al[e & 1];
                    }
                }
    #pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (!kFull && j == 1 && !two) break;
                    // this lane's four tokens of V, 8 dimensions each
                    const uint8_t* vb = st[j] + kSliceBytes + 8 * gq;
                    const uint2 v0 = *reinterpret_cast<const uint2*>(vb + vt0 * kHeadDim);
                    const uint2 v1 = *reinterpret_cast<const uint2*>(vb + vt1 * kHeadDim);
                    const uint2 v2 = *reinterpret_cast<const uint2*>(vb + (vt0 + 8) * kHeadDim);
                    const uint2 v3 = *reinterpret_cast<const uint2*>(vb + (vt1 + 8) * kHeadDim);
                    // the weights' bound and the size of the page's products, for each head
                    float bound[NT][2], size[NT][2];
                    const int byte = word[j] ? (int)(word[j] >> 16) : eo;  // (a page that is not there counts for nothing)
                    const bool own = !kFull && byte > *least + kSpread;
                    if (own) {  // weights relative to the page's own largest; products joined in 32 bits
    #pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
    #pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float m = fmaxf(x[j][nt][e], x[j][nt][2 + e]);
    #pragma unroll
                                for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                                bound[nt][e] = m;
                                size[nt][e] = m == kNegInf ? 0.f : fast_exp2(m - R[nt][e]);
                            }
                    } else {
                        if (!kFull && (unsigned)(byte - eo + kWindow) > 2u * kWindow) {  // O takes the page's value scale
                            const float f = q8::power(eo - byte);
    #pragma unroll
                            for (int mt = 0; mt < 4; ++mt)
    #pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
    #pragma unroll
                                    for (int e = 0; e < 4; ++e) O[mt][nt][e] *= f;
                            eo = byte;
                            *least = min(*least, eo - kWindow);
                        }
    #pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
    #pragma unroll
                            for (int e = 0; e < 2; ++e) bound[nt][e] = R[nt][e];
                    }
                    const int lift = kFull ? up[j] : own ? 0 : byte - eo;
                    const float vinv = q8::power(-lift), evl = (float)lift + kLift;
                    uint32_t pb[NT][2];
    #pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        // (a bound of -inf: no key seen yet, and none here: every x is -inf)
                        const float off0 = bound[nt][0] == kNegInf ? 0.f : evl - bound[nt][0];
                        const float off1 = bound[nt][1] == kNegInf ? 0.f : evl - bound[nt][1];
                        const float p0 = fast_exp2(x[j][nt][0] + off0), p2 = fast_exp2(x[j][nt][2] + off0);
                        const float p1 = fast_exp2(x[j][nt][1] + off1), p3 = fast_exp2(x[j][nt][3] + off1);
                        d[nt][0] += (p0 + p2) * (own ? size[nt][0] : vinv);
                        d[nt][1] += (p1 + p3) * (own ? size[nt][1] : vinv);
                        pb[nt][0] = movmatrix_trans(pack_f16(p0, p1));  // rows 0..7  -> B rows k = 2tq, 2tq+1
                        pb[nt][1] = movmatrix_trans(pack_f16(p2, p3));  // rows 8..15
                    }
                    // O^T += V^T P^T : tile mt holds dimensions 8 gq + 2 mt (row gq) and 8 gq + 2 mt + 1 (row gq + 8)
    #pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t a0 = h ? v0.y : v0.x, a1 = h ? v1.y : v1.x, a2 = h ? v2.y : v2.x, a3 = h ? v3.y : v3.x;
    #pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t sel = i ? 0x7362 : 0x5140;
                            const uint32_t lo = __byte_perm(a0, a1, sel), hi = __byte_perm(a2, a3, sel);
                            const uint32_t af[4] = {q8::f16x2_of(lo), q8::f16x2_of_high(lo), q8::f16x2_of(hi), q8::f16x2_of_high(hi)};
    #pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                float (&o)[4] = O[2 * h + i][nt];
                                if (own) {
                                    const float f = q8::power(byte - eo);
                                    float part[4] = {0.f, 0.f, 0.f, 0.f};
                                    mma_f16_16816(part, af, pb[nt][0], pb[nt][1]);
    #pragma unroll
                                    for (int e = 0; e < 4; ++e) o[e] += part[e] * f * size[nt][e & 1];
                                } else {
                                    mma_f16_16816(o, af, pb[nt][0], pb[nt][1]);
                                }
                            }
                        }
                    }
                }
            };
            if (calm && two && valid_of(0) == kPageSize && valid_of(1) == kPageSize) {
                pages(std::true_type{});
            } else {
                if (word[0]) *least = min(*least, (int)(word[0] >> 16));
                if (word[1]) *least = min(*least, (int)(word[1] >> 16));
                pages(std::false_type{});
            }

            // release the stages and refill them
            fence_proxy_async_smem();
            __syncwarp();
            consumed += two ? 2 : 1;
            if (more && issued - consumed <= kStages - 2) more = issue();
            if (more && issued - consumed <= kStages - 2) more = issue();
        }

        // ---- end of the piece: this warp's sum over its lanes
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) d[nt][e] += __shfl_xor_sync(0xffffffffu, d[nt][e], o);

        const float unit = q8::power(eo - kScaleBias);  // (of a piece without pages: O is 0)
        const long long slot = cta + seg;  // partial slot of this piece
        if (!cp.split()) {
            if (cnt > 0) {
                // one warp holds the whole piece: normalise, join the sink, write
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int h = nt * 8 + 2 * tq + e;
                        if (h >= G) continue;
                        const float dt = d[nt][e];
                        const float keys = dt > 0.f ? R[nt][e] - kLift + log2f(dt) : (dt == 0.f ? kNegInf : dt);
                        const float all = first ? log2_sum(keys, __ldg(&a.sinks[cp.g * G + h]) * kLog2e) : keys;
                        const float f = dt == 0.f ? 0.f : exp2f(keys - all) / dt * unit;
                        float v[8];
#pragma unroll
                        for (int mt = 0; mt < 4; ++mt) {
                            v[2 * mt] = dt == 0.f ? 0.f : O[mt][nt][e] * f;
                            v[2 * mt + 1] = dt == 0.f ? 0.f : O[mt][nt][2 + e] * f;
                        }
                        const long long row = (long long)cp.b * a.Hq + cp.g * G + h;
                        if (whole) {
                            reinterpret_cast<uint4*>(a.out + row * kHeadDim)[gq] =
                                make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
                        } else {
                            float4* dst = reinterpret_cast<float4*>(a.part_o + (slot * G + h) * kHeadDim + 8 * gq);
                            dst[0] = make_float4(v[0], v[1], v[2], v[3]);
                            dst[1] = make_float4(v[4], v[5], v[6], v[7]);
                        }
                        if (gq == 0) {
                            if (whole) {
                                if (a.lse) a.lse[row] = all * kLn2;
                            } else {
                                a.part_lse[slot * G + h] = all;
                            }
                        }
                    }
                }
            }
        } else {
            // ---- a dealt piece: drop this warp's state into the piece's combine slot; the last
            // warp to count itself in combines the states and writes the result
            const int sl = nsplit & 1, gen = nsplit >> 1;
            ++nsplit;
            if (!wait_word(&slot_gen[sl], gen)) {  // the slot's previous piece is combined
                failed = true;
                if (lane == 0) atomicOr(a.err, kErrTimeout);
            }
            __threadfence_block();
            float* co = cmb_o + sl * (kWarps * L::kHeads * kHeadDim);
            float* cmd = cmb_md + sl * (kWarps * L::kHeads * 2);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int h = nt * 8 + 2 * tq + e;
                    float4* dst = reinterpret_cast<float4*>(co + (warp * L::kHeads + h) * kHeadDim + 8 * gq);
                    dst[0] = make_float4(O[0][nt][e] * unit, O[0][nt][2 + e] * unit, O[1][nt][e] * unit, O[1][nt][2 + e] * unit);
                    dst[1] = make_float4(O[2][nt][e] * unit, O[2][nt][2 + e] * unit, O[3][nt][e] * unit, O[3][nt][2 + e] * unit);
                    if (lane < 4) {
                        cmd[(warp * L::kHeads + h) * 2 + 0] = R[nt][e];
                        cmd[(warp * L::kHeads + h) * 2 + 1] = d[nt][e];
                    }
                }
            }
            __syncwarp();
            int before = 0;
            if (lane == 0) {
                __threadfence_block();  // this warp's state is written before it counts itself in
                before = atomicAdd(&slot_arr[sl], 1);
                __threadfence_block();  // ... and the other warps' states are read after
            }
            before = __shfl_sync(0xffffffffu, before, 0);
            __syncwarp();
            if (before == kWarps - 1) {
                // the lanes split the G x 64 outputs: kLanesPerHead lanes per head, each with a run
                // of kDims consecutive head-dims, all loads of a run issued together
                constexpr int kLanesPerHead = 32 / L::kHeads;    // 4 (NT = 1) or 2 (NT = 2)
                constexpr int kDims = kHeadDim / kLanesPerHead;  // 16 or 32
                const int h = lane / kLanesPerHead, d0 = (lane % kLanesPerHead) * kDims;
                if (h < G) {
                    float sw[kWarps], M = kNegInf;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        sw[w] = cmd[(w * L::kHeads + h) * 2];
                        M = fmaxf(M, sw[w]);
                    }
                    float dt = 0.f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        sw[w] = (M == kNegInf || sw[w] == kNegInf) ? 0.f : fast_exp2(sw[w] - M);
                        dt += sw[w] * cmd[(w * L::kHeads + h) * 2 + 1];
                    }
                    const float keys = dt > 0.f ? M - kLift + log2f(dt) : (dt == 0.f ? kNegInf : dt);
                    const float all = first ? log2_sum(keys, __ldg(&a.sinks[cp.g * G + h]) * kLog2e) : keys;
                    const float f = dt == 0.f ? 0.f : exp2f(keys - all) / dt;
                    const long long row = (long long)cp.b * a.Hq + cp.g * G + h;
#pragma unroll
                    for (int part = 0; part < kDims / 8; ++part) {  // 8 head-dims at a time
                        float acc[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) acc[i] = 0.f;
#pragma unroll
                        for (int w = 0; w < kWarps; ++w) {
                            const float4* src =
                                reinterpret_cast<const float4*>(co + (w * L::kHeads + h) * kHeadDim + d0 + 8 * part);
                            const float4 v0 = src[0], v1 = src[1];
                            acc[0] += sw[w] * v0.x;
                            acc[1] += sw[w] * v0.y;
                            acc[2] += sw[w] * v0.z;
                            acc[3] += sw[w] * v0.w;
                            acc[4] += sw[w] * v1.x;
                            acc[5] += sw[w] * v1.y;
                            acc[6] += sw[w] * v1.z;
                            acc[7] += sw[w] * v1.w;
                        }
                        if (whole) {
                            reinterpret_cast<uint4*>(a.out + row * kHeadDim + d0)[part] =
                                make_uint4(pack_bf16(acc[0] * f, acc[1] * f), pack_bf16(acc[2] * f, acc[3] * f),
                                           pack_bf16(acc[4] * f, acc[5] * f), pack_bf16(acc[6] * f, acc[7] * f));
                        } else {
                            float4* dst = reinterpret_cast<float4*>(a.part_o + (slot * G + h) * kHeadDim + d0 + 8 * part);
                            dst[0] = make_float4(acc[0] * f, acc[1] * f, acc[2] * f, acc[3] * f);
                            dst[1] = make_float4(acc[4] * f, acc[5] * f, acc[6] * f, acc[7] * f);
                        }
                    }
                    if (d0 == 0) {
                        if (whole) {
                            if (a.lse) a.lse[row] = all * kLn2;
                        } else {
                            a.part_lse[slot * G + h] = all;
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) {  // free the slot for the piece after next
                    slot_arr[sl] = 0;
                    __threadfence_block();
                    *reinterpret_cast<volatile int*>(&slot_gen[sl]) = gen + 1;
                }
            }
        }
        cp = np;
        if (cp.ps < x1) cur = nxt;
    }

    if (failed) {
        // let copies already in flight land (bounded) before the CTA's shared memory is released
        for (int j = consumed; j < issued; ++j) (void)mbar_wait(&my_bars[j % kStages], (j / kStages) & 1);
    }

    // ---- 5. list the segment whose page 0 this share holds but does not complete: the merge
    // kernel combines its pieces (slots cta + seg .. cta + pieces - 1 + seg)
    if (tid == 0 && a.merge_list) {
        int2 e = make_int2(-1, 0);
        if (head_seg >= 0) {
            const int b = head_seg / Hkv, g = head_seg - b * Hkv;
            const int n = prefix[b + 1] - prefix[b];
            long long c_first;
            int pieces;
            segment_pieces((long long)prefix[b] * Hkv + (long long)g * n, n, C, U, c_first, pieces);
            e = make_int2(head_seg, pieces);
        }
        a.merge_list[cta] = e;
    }
}

const void* kernel_of(int NT) {
    return NT == 1 ? reinterpret_cast<const void*>(decode_q8_kernel<1>) : reinterpret_cast<const void*>(decode_q8_kernel<2>);
}

// Resident CTAs per SM x SM count for one (device, group width, shared memory) triple, remembered so that
// repeated calls skip the occupancy query.
cudaError_t resident_ctas_q8(int NT, size_t smem, long long* ctas) {
    struct Entry {
        int dev, NT;
        size_t smem;
        long long ctas;
    };
    static thread_local Entry cache[8] = {};
    static thread_local int next = 0;
    static thread_local bool done[2][64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    for (const Entry& c : cache)
        if (c.ctas > 0 && c.dev == dev && c.NT == NT && c.smem == smem) {
            *ctas = c.ctas;
            return cudaSuccess;
        }
    if ((e = allow_all_smem(kernel_of(NT), dev, done[NT - 1])) != cudaSuccess) return e;
    int sms = 0, per_sm = 0;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel_of(NT), kWarps * 32, smem)) != cudaSuccess) return e;
    if (per_sm < 1) return cudaErrorInvalidConfiguration;
    cache[next] = Entry{dev, NT, smem, (long long)sms * per_sm};
    next = (next + 1) % 8;
    *ctas = (long long)sms * per_sm;
    return cudaSuccess;
}

}  // namespace

cudaError_t decode_q8_plan(int B, int Hq, int Hkv, int num_workers, DecodeQ8Plan* plan) {
    const int G = Hq / Hkv;
    const int NT = G <= 8 ? 1 : 2;
    const size_t smem = (NT == 1 ? SmemLayout<1>::fixed : SmemLayout<2>::fixed) + size_t(B + 1) * 4;
    long long resident = 0;
    cudaError_t e = resident_ctas_q8(NT, smem, &resident);
    if (e != cudaSuccess) return e;
    const long long shares = num_workers > 0 ? num_workers : resident;
    plan->workers = (int)shares;
    plan->min_pages = SINKATTN_DECODE_Q8_MIN_PAGES;
    plan->grid = (int)shares;
    plan->smem = smem;
    plan->slots = (size_t)shares + (size_t)B * Hkv;
    size_t bytes = plan->slots * G * kHeadDim * 4;  // partial o
    bytes += plan->slots * G * 4;                   // partial lse (base 2)
    plan->merge_list_offset = (bytes + 255) & ~size_t(255);
    plan->ws_bytes = plan->merge_list_offset + (size_t)shares * sizeof(int2);
    return cudaSuccess;
}

cudaError_t decode_q8_launch(const DecodeQ8Args& args, const DecodeQ8Plan& plan, bool may_split, cudaStream_t stream) {
    if (args.B == 0) return cudaSuccess;
    DecodeQ8Args a = args;
    if (!may_split) a.merge_list = nullptr;
    // both kernels are programmatic dependents of what precedes them on the stream (decode.cu)
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)plan.grid);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = plan.smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = a.G <= 8 ? cudaLaunchKernelEx(&cfg, decode_q8_kernel<1>, a) : cudaLaunchKernelEx(&cfg, decode_q8_kernel<2>, a);
    if (e != cudaSuccess || !may_split) return e;
    SplitMergeArgs m;
    m.part_o = a.part_o;
    m.part_lse = a.part_lse;
    m.list = a.merge_list;
    m.out = a.out;
    m.lse = a.lse;
    m.listed = plan.grid;
    m.R = a.G;
    m.G = a.G;
    m.QL = 1;
    m.Hq = a.Hq;
    m.Hkv = a.Hkv;
    return split_merge_launch(m, stream);
}

}  // namespace sinkattn
