// decode_beams.cu -- decode of groups of rows (beams, or samples of one prompt) whose page tables share
// pages, on the fifth-generation tensor cores.
//
// The attention is the sink attention of "GPT-OSS on day 0" (Perplexity), section "Kernels for GPT-OSS / Sink
// Attention", of one query token per row over the row's own pages; the posts describe no sharing of pages
// between rows.  Softmax over a row's keys can be summed in any order and in any pieces, so the pages of a group
// are taken not row by row but once each: every distinct (column, page) with the set of rows that hold it.
//
// GB300 design.  beams_plan_kernel lists each group's distinct pages (its time is
// latency: a few dependent loads); decode_beams_kernel, its programmatic dependent, streams them.  The R = K x G
// query rows of one (group n, KV head g) -- row r = k * G + h is row k's query head g * G + h -- form ONE tcgen05
// tile (R <= 128, padded to the MMA's 128 rows), so a page is read once for all rows and every product runs on
// the tensor core; a row's keys are masked by the page's row set and the row's own length.
// Work: the flattened list of (group, KV head, 8 distinct pages = 128 keys) units, one contiguous share per CTA
// (one CTA per resident slot), cut at segment ends into pieces (the split of split_kv.cuh with tiles as units).
// The pipeline runs on across the pieces of a share:
//   warps 0, 3  TMA producers: warp 0 loads each piece's Q rows with one 3-D copy (64 dims x G heads x K rows,
//               landing as rows k * G + h) into a 2-slot Q ring and the K tiles, warp 3 the V tiles; a tile is 8
//               page copies of 2 KB (lanes 0-7), 128-byte swizzle.
//   warp 1      allocates 256 TMEM columns; issues S_j = Q K_j^T.
//   warp 2      issues O += P_j V_j (P read from TMEM; the first tile of a piece starts O afresh).
//   warps 4-7   softmax, thread r = row r (only the warps that hold rows work); at a piece's end they read O and
//               write the rows (or fp32 partials).
// A row fills a quarter or half of the tile's rows where R allows it: the query rows are then loaded two or four
// times, every copy takes its half or quarter of a tile's keys (the other keys' weights stay zero, so the products
// keep their form) and a state of its own, and the copies' states are put together at a piece's end.  All four
// softmax warps work then: 4 groups of 8 rows of 8 heads with 131072 tokens take 176 us, with one copy 201; 4 rows 168 and 180.
// A row's own pages are weights of zero for every other row of the group: a warp whose rows see none of its keys of a
// tile takes no maximum and no exponential of them.
// A weight of zero times a NaN or an infinity in such a page is a NaN in rows that do not hold it: rows whose sums come
// out not finite are taken again one by one at the share's end (out of line: in line its registers cost the whole 3 us).
// The piece with a segment's first tile is seeded with the sink.  The pieces of a segment split between CTAs
// write fp32 partials; the CTA holding the segment's first piece lists it, and the split-merge kernel, launched
// right behind this one as a programmatic dependent, combines them (merging in the CTA that finishes a segment's last
// piece takes longer: the fences that order its partials before the count wait for the copies in flight; 76 us against
// 57 for 32 groups of 8 rows).  Every wait is bounded.
//
// Measured (GB300, 64 query and 8 KV heads, calls back to back from a graph): 4 groups of 8 rows with 131072 tokens
// 176 us, 6.2 TB/s = 92% of the copy rate (HBM); sinkattn_decode on the 32 rows takes 686 us (8.6 GB of pages, many of them
// from L2).  4 rows a group, four copies of the query rows: 168 us, 95%.  32 groups of 8 rows with 512 to 4096 tokens, 128 of them
// a row's own, 54 us against 30.1 of reading (sinkattn_decode on the 256 rows 132 us): the tiles stream at the copy rate (20 of
// 1.5 us a CTA), but 11 us pass before the first scores (the plan 4, its end to the shares' start 4, the first pages 3),
// some 3 us at each piece's end, and the merge takes about 5.  More than 64 query rows: 16 rows a group 85 us against
// 39.3 of reading, the softmax's instructions (one thread a row and all 128 keys, two warps a scheduler).
#include "args_beams.h"
#include "args_merge.h"
#include "ptx.cuh"
#include "split_kv.cuh"
#include "tc_tile.cuh"

#include <cooperative_groups.h>

namespace cg = cooperative_groups;

namespace sinkattn {
namespace {

using namespace tc;

constexpr int kThreads = 256;
constexpr uint32_t kTmemCols = 256;
constexpr uint32_t kColS = 0, kColO = 128, kColP = 192;
constexpr int kKStages = 2, kVStages = 2;
constexpr int kPagesPerTile = kBN / kPageSize;  // 8
constexpr int kMinTiles = kBeamsMinTiles;  // automatic mode: never cut shares finer than this

constexpr int kPlanSteps = 8;  // columns of a lane in one pass

// Lists the distinct pages of group blockIdx.x / ctas, by column and, within one, by the first row that holds
// them; the group's CTAs are a cluster.  LANES neighbouring lanes take a column, one row each, so that one match over
// the warp finds every row's fellows, and a warp `steps` times 32 / LANES columns one after another, with all their
// loads issued first; the counts of the CTA's warps and of the cluster's CTAs then say where its entries go.
template <int LANES>
__global__ void __launch_bounds__(1024) beams_plan_kernel(const BeamsArgs a, const int steps) {
    __shared__ int len[kBeamsMaxBeams];
    __shared__ int red[32];
    __shared__ int counted[2];
    cg::cluster_group cluster = cg::this_cluster();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int kCols = 32 / LANES;  // columns of a warp's step
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = (int)blockDim.x / 32;
    const int K = a.K, cap = a.max_pages * kPageSize, k = lane % LANES, sub = lane / LANES;
    const int ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank(), n = (int)(blockIdx.x / (unsigned)ctas);
    int mine = 0;  // this lane's row's cached tokens
    if (k < K) {
        const int raw = __ldcg(&a.kv_lens[(long long)n * K + k]);
        if ((raw < 0 || raw > cap) && rank == 0 && warp == 0 && sub == 0) atomicOr(a.err, kErrBadLength);
        mine = clamp_len(raw, cap);
    }
    if (warp == 0 && sub == 0) len[k] = mine;
    const int longest = __reduce_max_sync(0xffffffffu, mine), shortest = __reduce_min_sync(0xffffffffu, k < K ? mine : cap);
    const int cols = (longest + kPageSize - 1) / kPageSize, held = (mine + kPageSize - 1) / kPageSize;  // held: by this row
    const int* row = a.page_table + ((long long)n * K + (k < K ? k : 0)) * a.max_pages;
    PageEntry* out = a.entries + (long long)n * K * a.max_pages;
    const unsigned fellows = LANES == 32 ? 0xffffffffu : ((1u << (LANES & 31)) - 1) << (sub * LANES);
    const int per = steps * kCols;  // columns of a warp's pass
    bool bad = false;
    int at = 0;
    for (long long q = 0, base = 0; base < cols; base += (long long)ctas * warps * per, ++q) {
        const long long c0 = base + (long long)(rank * warps + warp) * per + sub;
        int id[kPlanSteps];
#pragma unroll
        for (int s = 0; s < kPlanSteps; ++s) id[s] = s < steps && c0 + s * kCols < held ? __ldcg(&row[c0 + s * kCols]) : -1;
        unsigned same[kPlanSteps];  // the rows that hold this lane's page, for the first of them; else 0
        int count = 0;
#pragma unroll
        for (int s = 0; s < kPlanSteps; ++s) {
            same[s] = 0;
            if (s >= steps) continue;
            const bool there = id[s] >= 0 && id[s] < a.num_pages;
            bad |= !there && c0 + s * kCols < held;
            const unsigned all = __match_any_sync(0xffffffffu, there ? id[s] : ~lane) & fellows;
            if (there && __ffs(all) - 1 == lane) same[s] = all;
            count += __popc(__ballot_sync(0xffffffffu, same[s] != 0));
        }
        __syncthreads();
        if (lane == 0) red[warp] = count;
        __syncthreads();
        const int w = lane < warps ? red[lane] : 0;
        int total = __reduce_add_sync(0xffffffffu, w), to = at + __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
        if (ctas > 1) {
            if (tid == 0) counted[q & 1] = total;
            cluster.sync();
            total = 0;
            for (int i = 0; i < ctas; ++i) {
                const int there = cluster.map_shared_rank(counted, i)[q & 1];
                to += i < rank ? there : 0;
                total += there;
            }
        }
#pragma unroll
        for (int s = 0; s < kPlanSteps; ++s) {
            if (s >= steps) continue;
            const unsigned leaders = __ballot_sync(0xffffffffu, same[s] != 0);
            if (same[s]) {
                const int c = (int)c0 + s * kCols;
                const unsigned rows = same[s] >> (sub * LANES);
                int slots = kPageSize;
                if (shortest < (c + 1) * kPageSize) {  // how much of it the longest of its rows fills
                    slots = 0;
                    for (unsigned m = rows; m; m &= m - 1) slots = max(slots, min(kPageSize, len[__ffs(m) - 1] - c * kPageSize));
                }
                const bool all = __popc(rows) == K && shortest >= (c + 1) * kPageSize;
                *reinterpret_cast<int4*>(out + to + __popc(leaders & ((1u << lane) - 1))) =
                    make_int4(id[s], c, (int)rows, slots | (all ? kAllSee : 0));
            }
            to += __popc(leaders);
        }
        at += total;
    }
    if (bad) atomicOr(a.err, kErrBadPage);
    if (rank == 0 && tid == 0) a.counts[n] = at;
    if (ctas > 1) cluster.sync();  // no CTA ends while another reads its count
}

// What the plan kernel wrote is read through L2 (ld.cg): this kernel may be resident before it has been written.
__device__ __forceinline__ int count_of(const BeamsArgs& a, int n) { return __ldcg(&a.counts[n]); }
__device__ __forceinline__ int tiles_of(int pages) { return (pages + kPagesPerTile - 1) / kPagesPerTile; }
__device__ __forceinline__ PageEntry entry_of(const BeamsArgs& a, int n, int i) {
    const int4 e = __ldcg(reinterpret_cast<const int4*>(a.entries + (long long)n * a.K * a.max_pages + i));
    return PageEntry{e.x, e.y, (unsigned)e.z, e.w};
}

// One piece: tiles [ta, tb) of segment (b, g) (group b), whose first unit is seg_start and which has `tiles`
// tiles and `pages` distinct pages.
struct Piece {
    int b, g, ta, tb, tiles, pages;
    long long seg_start;
};

// The entry of lane l's page (l & 7) of tile t, or, where the segment has no such page, its last: read all the same, so
// that the load stays in flight until its value is needed (a choice made on the value would wait for it at once).
__device__ __forceinline__ int tile_entry(const Piece& p, int t, int lane) {
    const int i = t * kPagesPerTile + (lane & 7);
    return i < p.pages ? i : p.pages - 1;
}

// Walks the pieces of units [x, x1); every role of the CTA runs its own walker over the same share.
struct Walk {
    int b, g, tiles, pages;
    long long seg_start, x, x1;
    int B, Hkv;

    // the next segment with at least one tile (a walk never passes the share's end)
    __device__ void advance(const BeamsArgs& a) {
        seg_start += tiles;
        if (++g == Hkv) {
            g = 0;
            do {
                ++b;
                pages = count_of(a, b);
                tiles = tiles_of(pages);
            } while (tiles == 0 && b + 1 < B);
        }
    }
    __device__ bool next(const BeamsArgs& a, Piece& p) {
        if (x >= x1) return false;
        while (x >= seg_start + tiles) advance(a);
        p.b = b;
        p.g = g;
        p.tiles = tiles;
        p.pages = pages;
        p.seg_start = seg_start;
        p.ta = (int)(x - seg_start);
        const long long end = x1 < seg_start + tiles ? x1 : seg_start + tiles;
        p.tb = (int)(end - seg_start);
        x = end;
        return true;
    }
};

struct __align__(1024) Smem {
    uint8_t q[2][kTileBytes];
    uint8_t k[kKStages][kTileBytes];
    uint8_t v[kVStages][kTileBytes];
    uint64_t q_full[2], q_empty[2], k_full[kKStages], k_empty[kKStages], v_full[kVStages], v_empty[kVStages];
    uint64_t s_full, s_free, p_full, o_done, mma_done, exchange;
    uint32_t tmem_base;
    long long red[8];    // block reductions
    long long found[4];  // share start: group, its first unit, its pages, flag
    Walk walk[5];        // the softmax warps' walkers (kept out of their registers), and the share's start
    Piece piece[4];      // ... and their current pieces
    int4 entry[4][2][kPagesPerTile];  // the softmax warps' page entries, this tile's and the next one's
    float2 md[kBM];                   // SPLIT > 1: running maximum and normaliser of every thread at a piece's end
    float half[16][kBM];              // SPLIT = 4: the second exchange of partial sums
};

// The next piece of softmax warp `w`'s walk, found by its first lane; null at the end of the share.
__device__ __forceinline__ const Piece* next_piece(const BeamsArgs& a, Smem& sm, int w, int lane) {
    int has = 0;
    __syncwarp();  // every lane is done with the previous piece
    if (lane == 0) has = sm.walk[w].next(a, sm.piece[w]) ? 1 : 0;
    has = __shfl_sync(0xffffffffu, has, 0);
    __syncwarp();
    return has ? &sm.piece[w] : nullptr;
}

// cp.async of 16 bytes through L2, and the wait for all of a thread's.
__device__ __forceinline__ void copy16_async(void* smem, const void* gmem) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(smem)), "l"(gmem) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// One row's attention over its own pages among those of the piece, by a whole warp from global memory: the output's dims
// 2 lane and 2 lane + 1.  Two lanes take a slot's key, half of its dims each.
__device__ __forceinline__ float2 row_alone(const BeamsArgs& a, const Piece& pc, int row, int lane) {
    const int i = row / a.G, head = pc.g * a.G + row % a.G, slot = lane & 15;
    const long long beam = (long long)pc.b * a.K + i;
    const int len = clamp_len(__ldcg(&a.kv_lens[beam]), a.max_pages * kPageSize);
    const uint4* q = reinterpret_cast<const uint4*>(a.q + (beam * a.Hq + head) * kHeadDim) + 4 * (lane >> 4);
    float m = pc.ta == 0 ? __ldg(&a.sinks[head]) * kLog2e : kNegInf, d = pc.ta == 0 ? 1.f : 0.f;
    float2 sum = make_float2(0.f, 0.f);
    const int end = min(pc.pages, pc.tb * kPagesPerTile);
    for (int e = pc.ta * kPagesPerTile; e < end; ++e) {
        const PageEntry x = entry_of(a, pc.b, e);
        const int n = min(kPageSize, len - kPageSize * x.col);  // its keys in this page
        if (!((x.beams >> i) & 1u) || n <= 0) continue;
        const long long at = ((long long)x.page * a.Hkv + pc.g) * (kPageSize * kHeadDim);
        float dot = 0.f;
        if (slot < n) {
            const uint4* k = reinterpret_cast<const uint4*>(a.k_pages + at + slot * kHeadDim) + 4 * (lane >> 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint4 u = __ldcg(k + j), w = __ldcg(q + j);
                const uint32_t ku[4] = {u.x, u.y, u.z, u.w}, qw[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    dot = fmaf(__uint_as_float(ku[c] << 16), __uint_as_float(qw[c] << 16), dot);
                    dot = fmaf(__uint_as_float(ku[c] & 0xffff0000u), __uint_as_float(qw[c] & 0xffff0000u), dot);
                }
            }
        }
        dot += __shfl_xor_sync(0xffffffffu, dot, 16);
        const float s = slot < n ? dot * a.scale_log2 : kNegInf;
        float top = fmaxf(m, s);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float keep = m == kNegInf ? 0.f : fast_exp2(m - top), w = slot < n ? fast_exp2(s - top) : 0.f;
        m = top;
        float all = w;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
        d = d * keep + all;
        sum.x *= keep;
        sum.y *= keep;
        const uint32_t* v = reinterpret_cast<const uint32_t*>(a.v_pages + at) + lane;
#pragma unroll
        for (int j = 0; j < kPageSize; ++j) {
            const uint32_t u = j < n ? __ldcg(v + j * (kHeadDim / 2)) : 0u;
            const float wj = __shfl_sync(0xffffffffu, w, j);
            sum.x = fmaf(wj, __uint_as_float(u << 16), sum.x);
            sum.y = fmaf(wj, __uint_as_float(u & 0xffff0000u), sum.y);
        }
    }
    return d == 0.f ? make_float2(0.f, 0.f) : make_float2(sum.x / d, sum.y / d);
}

// The rows of a softmax warp whose sums in some piece of the share are not finite, taken again by themselves over the pages
// that they hold; `again` is the walk at the share's start.
template <int SPLIT>
__device__ __noinline__ void rows_alone(const BeamsArgs& a, Walk again) {
    constexpr int kBlock = kBM / SPLIT, kDims = kHeadDim / SPLIT;
    const int t0 = (int)threadIdx.x - 128, lane = t0 & 31, copy = t0 / kBlock, r = t0 % kBlock, R = a.R, G = a.G;
    const int dim0 = (SPLIT > 1 && (copy & 1) ? 32 : 0) + (SPLIT > 2 && (copy & 2) ? 16 : 0);
    Piece pc;
    while (again.next(a, pc)) {
        const bool whole = pc.ta == 0 && pc.tb == pc.tiles;
        const long long row0 = whole ? (long long)pc.b * a.K * a.Hq + pc.g * G
                                     : ((long long)blockIdx.x + pc.b * a.Hkv + pc.g) * R;
        auto place = [&](int row) {  // its first value in out or in the partials
            return (row0 + (whole ? (long long)(row / G) * a.Hq + row % G : row)) * kHeadDim;
        };
        bool redo = false;
        if (r < R) {
            const long long at = place(r) + dim0;
            for (int e = 0; e < kDims; ++e) {
                const float x = whole ? __bfloat162float(a.out[at + e]) : a.part_o[at + e];
                redo |= !(x * 0.f == 0.f);
            }
        }
        __syncwarp();
        for (unsigned left = __ballot_sync(0xffffffffu, redo); left; left &= left - 1) {
            const int from = __ffs(left) - 1, row = __shfl_sync(0xffffffffu, r, from);
            const int lo = __shfl_sync(0xffffffffu, dim0, from);
            const float2 x = row_alone(a, pc, row, lane);
            if (2 * lane < lo || 2 * lane >= lo + kDims) continue;
            const long long at = place(row) + 2 * lane;
            if (whole) *reinterpret_cast<uint32_t*>(a.out + at) = pack_bf16(x.x, x.y);
            else *reinterpret_cast<float2*>(a.part_o + at) = x;
        }
    }
}

template <int SPLIT>
__global__ void __launch_bounds__(kThreads, 2)
    decode_beams_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                     const __grid_constant__ CUtensorMap tmap_v, const BeamsArgs a) {
    extern __shared__ uint8_t smem_raw[];
    Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int B = a.N, Hkv = a.Hkv, R = a.R, K = a.K, G = a.G;
    constexpr int kKeys = kBN / SPLIT;  // keys of a tile that a softmax thread takes
    constexpr int kBlock = kBM / SPLIT;  // rows of a copy of the query rows
    constexpr int kBlocks = SPLIT == 1 ? kKeys / 32 : 1;  // parts of a thread's keys that are left out where no row sees them
    const int active = SPLIT > 1 ? 4 : (R + 31) / 32;  // softmax warps that hold rows

    // ---- 0. set-up that reads no input (barriers, tensor memory, the Q padding): done before the wait
    // below, so it overlaps the preceding kernel's tail
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.q_full[i], 1);
            mbar_init(&sm.q_empty[i], SPLIT > 1 ? 1 + 128 : 1);
        }
        for (int i = 0; i < kKStages; ++i) {
            mbar_init(&sm.k_full[i], 1);
            mbar_init(&sm.k_empty[i], 1);
        }
        for (int i = 0; i < kVStages; ++i) {
            mbar_init(&sm.v_full[i], 1);
            mbar_init(&sm.v_empty[i], 1);
        }
        mbar_init(&sm.s_full, 1);
        mbar_init(&sm.s_free, 32 * active);
        mbar_init(&sm.p_full, 32 * active);
        mbar_init(&sm.o_done, 1);
        mbar_init(&sm.mma_done, 2);
        mbar_init(&sm.exchange, 128);
        fence_mbar_init();
        fence_proxy_async_smem();
    }
    if (warp == 1) {
        tmem_alloc(&sm.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    // rows without a query start as zeros; the TMA writes the first R rows of every copy
    for (int e = tid; e < kBM * 8; e += kThreads) {
        if ((e >> 3) % kBlock < R) continue;
        reinterpret_cast<uint4*>(sm.q[0])[e] = make_uint4(0u, 0u, 0u, 0u);
        reinterpret_cast<uint4*>(sm.q[1])[e] = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();

    // a programmatic dependent of what precedes it on the stream: no input is read before that has
    // completed; the split merge behind this kernel may be scheduled once every CTA runs
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- 1. units (Hkv x tiles) per group: their total U and, by a running block-wide scan, the
    // group holding this share's first unit (one pass when the batch fits the CTA's threads)
    if (tid == 0) sm.found[3] = 0;
    long long U = 0, base = 0, lo = 0, cnt = 0;
    int pages_here = 0;
    for (int p0 = 0; p0 < B; p0 += kThreads) {
        const int i = p0 + tid;
        const int n_pages = i < B ? count_of(a, i) : 0, ti = tiles_of(n_pages);
        const long long c = (long long)ti * Hkv;
        long long incl = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        __syncthreads();  // red[] is free
        if (lane == 31) sm.red[warp] = incl;
        __syncthreads();
        long long woff = 0, total = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            woff += w < warp ? sm.red[w] : 0;
            total += sm.red[w];
        }
        if (B <= kThreads) {  // one pass: this thread's request and its units stay in registers
            lo = woff + incl - c;
            cnt = c;
            pages_here = n_pages;
        }
        U = base + total;
        base = U;
    }
    {  // rows of groups without a page carry only the sink
        const long long rows = (long long)B * K * a.Hq;
        for (long long r = (long long)blockIdx.x * kThreads + tid; r < rows; r += (long long)gridDim.x * kThreads) {
            const int b = (int)(r / ((long long)K * a.Hq));
            if (count_of(a, b) != 0) continue;
            uint4* dst = reinterpret_cast<uint4*>(a.out + r * kHeadDim);
#pragma unroll
            for (int e = 0; e < 8; ++e) dst[e] = make_uint4(0u, 0u, 0u, 0u);
            if (a.lse) a.lse[r] = __ldg(&a.sinks[r % a.Hq]);
        }
    }
    const long long C = U > 0 ? effective_shares(a.tc_grid, a.fixed_workers, kMinTiles, U) : 0;
    const long long cta = blockIdx.x;
    if (cta >= C) {  // no share: release the tensor memory taken above (the whole CTA is here)
        if (tid == 0 && a.merge_list) a.merge_list[cta] = make_int2(-1, 0);
        tc_fence_before();
        __syncthreads();
        if (warp == 1) {
            tc_fence_after();
            tmem_dealloc(sm.tmem_base, kTmemCols);
        }
        return;
    }
    const long long x0 = cta * U / C, x1 = (cta + 1) * U / C;
    if (B <= kThreads) {
        if (cnt > 0 && x0 >= lo && x0 < lo + cnt) {
            sm.found[0] = tid;
            sm.found[1] = lo;
            sm.found[2] = pages_here;
        }
        __syncthreads();
    } else {
        // ---- 2. a second scan, now that U (and so x0) is known
        base = 0;
        for (int p0 = 0; p0 < B; p0 += kThreads) {
            const int i = p0 + tid;
            const int n_pages = i < B ? count_of(a, i) : 0, ti = tiles_of(n_pages);
            const long long c = (long long)ti * Hkv;
            long long incl = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            __syncthreads();  // red[] (and found[3]) are settled
            if (lane == 31) sm.red[warp] = incl;
            __syncthreads();
            long long woff = 0, total = 0;
#pragma unroll
            for (int w = 0; w < kThreads / 32; ++w) {
                woff += w < warp ? sm.red[w] : 0;
                total += sm.red[w];
            }
            const long long l0 = base + woff + incl - c;
            if (c > 0 && x0 >= l0 && x0 < l0 + c) {
                sm.found[0] = i;
                sm.found[1] = l0;
                sm.found[2] = n_pages;
                sm.found[3] = 1;
            }
            base += total;
            __syncthreads();
            if (sm.found[3]) break;
        }
    }
    Walk walk;
    walk.B = B;
    walk.Hkv = Hkv;
    walk.b = (int)sm.found[0];
    walk.pages = (int)sm.found[2];
    walk.tiles = tiles_of(walk.pages);
    walk.g = (int)((x0 - sm.found[1]) / walk.tiles);
    walk.seg_start = sm.found[1] + (long long)walk.g * walk.tiles;
    walk.x = x0;
    walk.x1 = x1;
    if (tid < 5) sm.walk[tid] = walk;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = sm.tmem_base;

    if (warp < 4) {
        // 128 x kFew + 128 x kMany = 256 x 128, the launch's registers: a thread's scores of a whole tile want many
        constexpr int kFew = SPLIT > 1 ? 96 : 64;
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFew));
        if (warp == 0 || warp == 3) {
            // ------------------------------------------------------------ TMA producers
            const bool is_k = warp == 0;
            const int stages = is_k ? kKStages : kVStages;
            uint64_t* full = is_k ? sm.k_full : sm.v_full;
            uint64_t* empty = is_k ? sm.k_empty : sm.v_empty;
            const CUtensorMap* map = is_k ? &tmap_k : &tmap_v;
            if (lane == 0) {
                tma_prefetch_desc(map);
                if (is_k) tma_prefetch_desc(&tmap_q);
            }
            int J = 0, p = 0, issued = 0;  // tiles, pieces (their Q issued) and tile copies issued so far
            bool ok = true;
            Piece pc;
            while (ok && walk.next(a, pc)) {
                if (is_k) {  // this piece's Q rows into Q slot p & 1, once the piece two back has used it
                    int got = 1;
                    if (lane == 0) {
                        if (p >= 2) got = mbar_wait(&sm.q_empty[p & 1], ((p >> 1) - 1) & 1);
                        if (got) {
                            mbar_arrive_expect_tx(&sm.q_full[p & 1], (uint32_t)(SPLIT * R) * 128u);
#pragma unroll
                            for (int c = 0; c < SPLIT; ++c)
                                tma_load_3d(sm.q[p & 1] + c * kBlock * 128, &tmap_q, 0, pc.g * G, pc.b * K, &sm.q_full[p & 1]);
                        }
                    }
                    if (!(ok = __shfl_sync(0xffffffffu, got, 0) != 0)) break;
                }
                ++p;
                // page ids (lanes 0-7), read one tile ahead of the copies
                int page = entry_of(a, pc.b, tile_entry(pc, pc.ta, lane)).page;
                for (int t = pc.ta; ok && t < pc.tb; ++t, ++J) {
                    const int st = J % stages;
                    if (J >= stages) {
                        int got = 0;
                        if (lane == 0) got = mbar_wait(&empty[st], ((J / stages) - 1) & 1);
                        if (!(ok = __shfl_sync(0xffffffffu, got, 0) != 0)) break;
                    }
                    // a tile's missing pages are copied from behind the pool's end: zeros
                    const int row = t * kPagesPerTile + lane < pc.pages ? (page * Hkv + pc.g) * kPageSize
                                                                        : a.num_pages * Hkv * kPageSize;
                    page = entry_of(a, pc.b, tile_entry(pc, t + 1, lane)).page;
                    if (lane == 0) mbar_arrive_expect_tx(&full[st], kTileBytes);
                    __syncwarp();
                    uint8_t* tile = is_k ? sm.k[st] : sm.v[st];
                    if (lane < kPagesPerTile) tma_load_2d(tile + lane * (kPageSize * 128), map, 0, row, &full[st]);
                    issued = J + 1;
                }
            }
            if (is_k && lane == 0 && a.merge_list) {
                // list the segment whose first piece this share holds without completing it (its last piece, if any): the
                // split merge combines its partials once every CTA has finished
                int2 head = make_int2(-1, 0);
                if (ok && pc.ta == 0 && pc.tb < pc.tiles) {
                    long long c_first = 0;
                    int pieces = 0;
                    segment_pieces(pc.seg_start, pc.tiles, C, U, c_first, pieces);
                    head = make_int2(pc.b * Hkv + pc.g, pieces);
                }
                a.merge_list[cta] = head;
            }
            if (!ok && lane == 0) atomicOr(a.err, kErrTimeout);
            // every copy this warp started has landed before the CTA can exit (bounded)
            if (lane == 0) {
                for (int j = issued - stages < 0 ? 0 : issued - stages; j < issued; ++j)
                    (void)mbar_wait(&full[j % stages], (j / stages) & 1);
                if (is_k)
                    for (int q = p - 2 < 0 ? 0 : p - 2; q < p; ++q) (void)mbar_wait(&sm.q_full[q & 1], (q >> 1) & 1);
            }
        } else if (warp == 1) {
            // ------------------------------------------------------------ S issuer: S_j = Q K_j^T
            // (the whole warp walks the loop, one elected lane issues)
            const uint32_t tS = tbase + kColS;
            int J = 0, p = 0;
            bool ok = true;
            Piece pc;
            while (ok && walk.next(a, pc)) {
                if (!(ok = warp_wait(&sm.q_full[p & 1], (p >> 1) & 1))) break;
                const uint32_t qaddr = smem_u32(sm.q[p & 1]);
                for (int t = pc.ta; t < pc.tb; ++t, ++J) {
                    const int st = J % kKStages;
                    ok = warp_wait(&sm.k_full[st], (J / kKStages) & 1) && (J == 0 || warp_wait(&sm.s_free, (J - 1) & 1));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t kaddr = smem_u32(sm.k[st]);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        tc_mma_ss_warp(tS, sw128_desc(qaddr + kk * 32), sw128_desc(kaddr + kk * 32), kIdescQK, kk > 0);
                    tc_commit_warp(&sm.s_full);
                    tc_commit_warp(&sm.k_empty[st]);
                }
                tc_commit_warp(&sm.q_empty[p & 1]);  // this piece's Q slot is free once its products end
                ++p;
            }
            if (!ok && lane == 0) atomicOr(a.err, kErrTimeout);
            tc_commit_warp(&sm.mma_done);  // every MMA of both issuers has finished before TMEM is released
            (void)warp_wait(&sm.mma_done, 0);
        } else if (warp == 2) {
            // ------------------------------------------------------------ PV issuer: O += P_j V_j
            // One elected lane issues; the whole warp zeroes the slots of V that hold no token of any row (they
            // may hold anything, and a 0 weight times NaN is NaN) before a tile's product.
            const uint32_t tO = tbase + kColO, tP = tbase + kColP;
            int J = 0;
            bool ok = true;
            Piece pc;
            while (ok && walk.next(a, pc)) {
                int slots = entry_of(a, pc.b, tile_entry(pc, pc.ta, lane)).slots;  // read one tile ahead
                for (int t = pc.ta; t < pc.tb; ++t, ++J) {
                    const int st = J % kVStages;
                    ok = warp_wait(&sm.v_full[st], (J / kVStages) & 1);
                    if (!ok) break;
                    // (the slots of missing pages are zeros already)
                    const int filled = slots & ~kAllSee;
                    uint32_t part = __ballot_sync(0xffffffffu, lane < kPagesPerTile && t * kPagesPerTile + lane < pc.pages &&
                                                                   filled < kPageSize);
                    slots = entry_of(a, pc.b, tile_entry(pc, t + 1, lane)).slots;
                    if (part) {
                        while (part) {
                            const int pg = __ffs(part) - 1;
                            part &= part - 1;
                            const int n = __shfl_sync(0xffffffffu, filled, pg);
                            for (int e = (pg * kPageSize + n) * 8 + lane; e < (pg + 1) * kPageSize * 8; e += 32)
                                reinterpret_cast<uint4*>(sm.v[st])[e] = make_uint4(0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    if (!(ok = warp_wait(&sm.p_full, J & 1))) break;
                    tc_fence_after();
                    const uint32_t vaddr = smem_u32(sm.v[st]);
                    // P_j is written only after the softmax has read the previous piece's O, so the first tile of
                    // a piece may start O afresh
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        tc_mma_ts_warp(tO, tP + ks * 8, sw128_desc(vaddr + ks * 2048), kIdescPV,
                                       (t > pc.ta || ks > 0) ? 1u : 0u);
                    tc_commit_warp(&sm.v_empty[st]);
                    tc_commit_warp(&sm.o_done);
                }
            }
            if (!ok && lane == 0) atomicOr(a.err, kErrTimeout);
            tc_commit_warp(&sm.mma_done);
            (void)warp_wait(&sm.mma_done, 0);
        }
    } else {
        constexpr int kMany = SPLIT > 1 ? 160 : 192;
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kMany));
        const int copy = (tid - 128) / kBlock, r = (tid - 128) % kBlock;  // copy of the query rows, row
        const bool live = r < R;
        const int i = live ? r / G : 0, h = live ? r % G : 0;
        if (warp - 4 < active) {
            // ---------------------------------------------------------------- softmax
            const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
            const uint32_t tS = tbase + lane_off + kColS + copy * kKeys, tO = tbase + lane_off + kColO;
            const uint32_t tP = tbase + lane_off + kColP;
            const float scale_log2 = a.scale_log2;
            if constexpr (SPLIT > 1) {  // the weights of the keys that other copies take stay zero
                uint32_t zero[32] = {};
                tmem_st32(tP, zero);
                tmem_st32(tP + 32, zero);
                tc_wait_st();
            }
            auto store_p = [&](uint32_t (&pk)[kKeys / 2]) {
                if constexpr (SPLIT == 4) {
                    tmem_st16(tP + copy * 16, pk);
                } else {
#pragma unroll
                    for (int cc = 0; cc < kKeys / 64; ++cc)
                        tmem_st32(tP + copy * (kKeys / 2) + cc * 32, *reinterpret_cast<uint32_t(*)[32]>(&pk[cc * 32]));
                }
            };
            const uint32_t mine = live ? 1u << i : 0u;
            bool blank = SPLIT > 1;    // this warp's weights are zeros
            // the dims of its row that a thread finishes (see the exchange below)
            constexpr int kDims = kHeadDim / SPLIT;
            const int dim0 = (SPLIT > 1 && (copy & 1) ? 32 : 0) + (SPLIT > 2 && (copy & 2) ? 16 : 0);
            bool odd = false;          // a sum that is not finite
            int J = 0, p = 0, ex = 0;  // tiles, pieces, phases of the exchange barrier
            bool ok = true;
            const int sw = warp - 4;
            // the entries of a tile's pages are copied to shared memory one tile ahead (in registers they would not fit
            // beside the scores, and a spill waits for the load)
            const PageEntry* entries = nullptr;  // of the piece's group
            auto fetch = [&](int t, int pages) {
                const int e = t * kPagesPerTile + lane;
                if (lane < kPagesPerTile) copy16_async(&sm.entry[sw][t & 1][lane], entries + (e < pages ? e : pages - 1));
            };
            // a piece's first entries, and this row's cached tokens (the plan kernel reported lengths out of range)
            auto begin = [&](const Piece& pc) {
                entries = a.entries + (long long)pc.b * K * a.max_pages;
                fetch(pc.ta, pc.pages);
                return live ? __ldcg(&a.kv_lens[(long long)pc.b * K + i]) : 0;
            };
            const Piece* next = next_piece(a, sm, sw, lane);
            int cached = next ? begin(*next) : 0;
            while (next) {
                const Piece& pc = *next;
                const int ta = pc.ta, tb = pc.tb, pages = pc.pages, seg = pc.b * Hkv + pc.g;
                const bool starts = ta == 0, whole = starts && tb == pc.tiles;
                const int len = clamp_len(cached, a.max_pages * kPageSize);
                const bool seeded = starts && copy == 0;
                float m = (seeded && live) ? __ldg(&a.sinks[pc.g * G + h]) * kLog2e : kNegInf;
                float d = (seeded && live) ? 1.f : 0.f;  // the sink's own e^(sink - m) = 1
                for (int t = ta; t < tb; ++t, ++J) {
                    copies_done();
                    __syncwarp();
                    const int4* entry = sm.entry[sw][t & 1];
                    if (t + 1 < tb) fetch(t + 1, pages);
                    // does any row of this warp's keys' pages see less than all of them?
                    constexpr int kMine = kKeys / kPageSize;  // pages of this copy's keys
                    const int page0 = copy * kMine, left = pages - t * kPagesPerTile - page0;
                    const bool masked =
                        left < kMine || !__all_sync(0xffffffffu, (entry[page0 + lane % kMine].w & kAllSee) != 0);
                    // this row's visible keys: of each page, the slots its length reaches; `use`: the blocks of 32 keys of
                    // which some row of this warp sees any
                    uint32_t vis[kKeys / 32], use = ~0u;
                    if (masked) {
                        use = 0u;
#pragma unroll
                        for (int w = 0; w < kKeys / 32; ++w) {
                            vis[w] = 0u;
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                const int4 e = entry[page0 + 2 * w + half];
                                const int n = max(0, min(kPageSize, len - kPageSize * e.y));
                                const uint32_t bits = ((1u << n) - 1u) << (16 * half);
                                if (((uint32_t)e.z & mine) && 2 * w + half < left) vis[w] |= bits;
                            }
                            use |= __any_sync(0xffffffffu, vis[w] != 0u) ? 1u << w : 0u;
                        }
                    }
                    if (!(ok = warp_wait(&sm.s_full, J & 1))) break;
                    tc_fence_after();
                    const bool first = t == ta;  // O starts afresh with this piece
                    if (use == 0u) {  // pages of other warps' rows only: no weight changes
                        mbar_arrive(&sm.s_free);
                        if (!first) {
                            if (!(ok = warp_wait(&sm.o_done, (J - 1) & 1))) break;
                            tc_fence_after();
                        }
                        if (!blank) {
                            uint32_t zero[kKeys / 2] = {};
                            store_p(zero);
                            tc_wait_st();
                            blank = true;
                        }
                        tc_fence_before();
                        mbar_arrive(&sm.p_full);
                        continue;
                    }
                    float s[kKeys];
#pragma unroll
                    for (int cc = 0; cc < kKeys / 32; ++cc)
                        tmem_ld32(tS + cc * 32, *reinterpret_cast<uint32_t(*)[32]>(&s[cc * 32]));
                    tc_wait_ld();
                    tc_fence_before();
                    mbar_arrive(&sm.s_free);

                    float mul = scale_log2;
                    if (!(scale_log2 > 0.f)) {  // zero or negative scale: scale first, mask after
#pragma unroll
                        for (int cc = 0; cc < kKeys; ++cc) s[cc] *= scale_log2;
                        mul = 1.f;
                    }
                    if (masked && kBlocks == 1) {
#pragma unroll
                        for (int cc = 0; cc < kKeys; ++cc) s[cc] = ((vis[cc >> 5] >> (cc & 31)) & 1u) ? s[cc] : kNegInf;
                    }
                    constexpr int kPer = kKeys / kBlocks;
                    float mx_raw = kNegInf;
#pragma unroll
                    for (int w = 0; w < kBlocks; ++w) {
                        float* x = s + w * kPer;
                        if (kBlocks > 1) {
                            if (!((use >> w) & 1u)) continue;
                            if (masked) {
#pragma unroll
                                for (int cc = 0; cc < kPer; ++cc) x[cc] = ((vis[w] >> cc) & 1u) ? x[cc] : kNegInf;
                            }
                        }
                        float acc[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) acc[e] = fmax3(x[e], x[8 + e], x[16 + e]);
#pragma unroll
                        for (int cc = 24; cc < kPer - 8; cc += 16)
#pragma unroll
                            for (int e = 0; e < 8; ++e) acc[e] = fmax3(acc[e], x[cc + e], x[cc + 8 + e]);
#pragma unroll
                        for (int e = 0; e < 8; ++e) acc[e] = fmaxf(acc[e], x[kPer - 8 + e]);
                        mx_raw = fmaxf(mx_raw, fmaxf(fmax3(acc[0], acc[1], acc[2]),
                                                     fmax3(acc[3], acc[4], fmax3(acc[5], acc[6], acc[7]))));
                    }
                    const float mx = mx_raw == kNegInf ? kNegInf : mx_raw * mul;
                    const float m_new = fmaxf(m, mx);
                    float factor = 1.f;
                    bool rescale_o = false;
                    if (first || m_new > m + kRescaleThreshold) {
                        factor = (m_new == kNegInf) ? 1.f : fast_exp2(m - m_new);
                        rescale_o = !first;
                        m = m_new;
                        d *= factor;
                    }
                    const float neg_m = (m == kNegInf) ? 0.f : -m;
                    const float2 mul2 = make_float2(mul, mul), negm2 = make_float2(neg_m, neg_m);
                    float2 sums[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                                      make_float2(0.f, 0.f)};
                    uint32_t pk[kKeys / 2];
#pragma unroll
                    for (int w = 0; w < kKeys / 32; ++w) {
                        if (kBlocks == 1 || ((use >> w) & 1u)) {
#pragma unroll
                            for (int cc = 16 * w; cc < 16 * w + 16; ++cc) {
                                const float2 xx = ffma2(make_float2(s[2 * cc], s[2 * cc + 1]), mul2, negm2);
                                const float2 pp = make_float2(fast_exp2(xx.x), fast_exp2(xx.y));
                                sums[cc & 3] = fadd2(sums[cc & 3], pp);
                                pk[cc] = pack_bf16(pp.x, pp.y);
                            }
                        } else {
#pragma unroll
                            for (int cc = 16 * w; cc < 16 * w + 16; ++cc) pk[cc] = 0u;
                        }
                    }
                    const float2 s01 = fadd2(fadd2(sums[0], sums[1]), fadd2(sums[2], sums[3]));
                    d += s01.x + s01.y;
                    if (!first) {  // P_{j-1} consumed and O_{j-1} final before P and O are touched
                        if (!(ok = warp_wait(&sm.o_done, (J - 1) & 1))) break;
                        tc_fence_after();
                        if (__any_sync(0xffffffffu, rescale_o)) {
#pragma unroll
                            for (int cc = 0; cc < 2; ++cc) {
                                uint32_t o[32];
                                tmem_ld32(tO + cc * 32, o);
                                tc_wait_ld();
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * factor);
                                tmem_st32(tO + cc * 32, o);
                            }
                        }
                    }
                    store_p(pk);
                    blank = false;
                    tc_wait_st();
                    tc_fence_before();
                    mbar_arrive(&sm.p_full);
                }
                if (!ok) break;
                const long long row0 = (long long)pc.b * K * a.Hq + pc.g * G;
                // the next piece is looked up while the last product runs
                next = next_piece(a, sm, sw, lane);
                if (next) cached = begin(*next);
                // ---- end of the piece (the PV of its last tile has finished): O / d of this row
                if (!(ok = warp_wait(&sm.o_done, (J - 1) & 1))) break;
                tc_fence_after();
                uint32_t raw[64];
                tmem_ld32(tO, *reinterpret_cast<uint32_t(*)[32]>(&raw[0]));
                tmem_ld32(tO + 32, *reinterpret_cast<uint32_t(*)[32]>(&raw[32]));
                tc_wait_ld();
                tc_fence_before();
                float o[64];
#pragma unroll
                for (int e = 0; e < 64; ++e) o[e] = __uint_as_float(raw[e]);
                float scale_o = d > 0.f ? 1.f / d : 0.f, l2 = d > 0.f ? m + log2f(d) : kNegInf;
                if constexpr (SPLIT > 1) {
                    // the copies' sums of a row, brought to one maximum, are added up: each thread gives the dims that it
                    // does not finish to the thread of the same row in another copy
                    // (through the piece's Q slot, which is free: its scores are done)
                    const int t0 = tid - 128;
                    float(*give)[kBM] = reinterpret_cast<float(*)[kBM]>(sm.q[p & 1]);
                    const bool upper = copy & 1;
                    sm.md[t0] = make_float2(m, d);
#pragma unroll
                    for (int e = 0; e < 32; ++e) give[e][t0] = upper ? o[e] : o[32 + e];
                    mbar_arrive(&sm.exchange);
                    if (!(ok = warp_wait(&sm.exchange, ex++ & 1))) break;
                    float M = m, D = 0.f;
#pragma unroll
                    for (int c = 0; c < SPLIT; ++c) M = fmaxf(M, sm.md[c * kBlock + r].x);
#pragma unroll
                    for (int c = 0; c < SPLIT; ++c) {
                        const float2 x = sm.md[c * kBlock + r];
                        D += x.x == kNegInf ? 0.f : x.y * fast_exp2(x.x - M);
                    }
                    // (all mass on nothing: a sink of -inf and no key)
                    l2 = D > 0.f ? M + log2f(D) : kNegInf;
                    auto share = [&](float mc) { return (mc == kNegInf || !(D > 0.f)) ? 0.f : fast_exp2(mc - M) / D; };
                    const float ours = share(m), theirs = share(sm.md[t0 ^ kBlock].x);
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = (upper ? o[32 + e] : o[e]) * ours + give[e][t0 ^ kBlock] * theirs;
                    scale_o = 1.f;
                    fence_proxy_async_smem();  // before a copy of query rows may land there
                    mbar_arrive(&sm.q_empty[p & 1]);
                    if constexpr (SPLIT == 4) {
                        const bool upper2 = copy & 2;
#pragma unroll
                        for (int e = 0; e < 16; ++e) sm.half[e][t0] = upper2 ? o[e] : o[16 + e];
                        mbar_arrive(&sm.exchange);
                        if (!(ok = warp_wait(&sm.exchange, ex++ & 1))) break;
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = (upper2 ? o[16 + e] : o[e]) + sm.half[e][t0 ^ (2 * kBlock)];
                    }
                    ++p;
                }
                float probe = 0.f;  // a NaN if any of the sums is not finite
#pragma unroll
                for (int e = 0; e < kDims; ++e) probe = fmaf(o[e], 0.f, probe);
                odd |= live && probe * scale_o != 0.f;
                if (live) {
                    if (whole) {
                        const long long row = row0 + (long long)i * a.Hq + h;
                        uint4* dst = reinterpret_cast<uint4*>(a.out + row * kHeadDim + dim0);
#pragma unroll
                        for (int e = 0; e < kDims / 8; ++e) {
                            uint4 w;
                            w.x = pack_bf16(o[8 * e + 0] * scale_o, o[8 * e + 1] * scale_o);
                            w.y = pack_bf16(o[8 * e + 2] * scale_o, o[8 * e + 3] * scale_o);
                            w.z = pack_bf16(o[8 * e + 4] * scale_o, o[8 * e + 5] * scale_o);
                            w.w = pack_bf16(o[8 * e + 6] * scale_o, o[8 * e + 7] * scale_o);
                            dst[e] = w;
                        }
                        if (a.lse && copy == 0) a.lse[row] = l2 * kLn2;
                    } else {
                        const long long slot = cta + seg;  // partial slot of this piece
                        float4* dst = reinterpret_cast<float4*>(a.part_o + (slot * R + r) * kHeadDim + dim0);
#pragma unroll
                        for (int e = 0; e < kDims / 4; ++e)
                            dst[e] = make_float4(o[4 * e + 0] * scale_o, o[4 * e + 1] * scale_o, o[4 * e + 2] * scale_o,
                                                 o[4 * e + 3] * scale_o);
                        if (copy == 0) a.part_lse[slot * R + r] = l2;
                    }
                }
            }
            copies_done();
            // a weight of zero times a NaN or infinity in another row's page is a NaN (nothing waits for this warp any
            // more but the CTA's end)
            if (ok && __any_sync(0xffffffffu, odd)) rows_alone<SPLIT>(a, sm.walk[4]);
            if (!ok && lane == 0) atomicOr(a.err, kErrTimeout);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tbase, kTmemCols);
    }
}

}  // namespace

// The kernel for R query rows: as many copies of them as the tile's 128 rows hold, so that all four softmax warps work.
using BeamsKernel = void (*)(const CUtensorMap, const CUtensorMap, const CUtensorMap, const BeamsArgs);
static BeamsKernel beams_kernel(int R, int* split) {
    *split = R <= 32 ? 4 : (R <= 64 ? 2 : 1);
    return R <= 32 ? decode_beams_kernel<4> : (R <= 64 ? decode_beams_kernel<2> : decode_beams_kernel<1>);
}

// CTAs of the attention kernel that fit on one SM, from its registers, its shared memory (with the per-block
// reservation) and its tensor memory (512 columns per SM, kTmemCols per CTA); the runtime's occupancy query
// reports one for a kernel that allocates tensor memory, while the hardware keeps two resident.
static cudaError_t beams_occupancy(int R, int* per_sm, int* sms) {
    static thread_local int cached[64][5] = {};
    int dev = 0, split = 1;
    const BeamsKernel kernel = beams_kernel(R, &split);
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    if (dev < 64 && cached[dev][split] > 0) {
        *per_sm = cached[dev][split];
        return cudaSuccess;
    }
    const size_t smem = 1024 + sizeof(Smem);
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, kernel)) != cudaSuccess) return e;
    int smem_sm = 0, reserved = 0, regs_sm = 0;
    if ((e = cudaDeviceGetAttribute(&smem_sm, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&reserved, cudaDevAttrReservedSharedMemoryPerBlock, dev)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&regs_sm, cudaDevAttrMaxRegistersPerMultiprocessor, dev)) != cudaSuccess)
        return e;
    const int regs_warp = ((fa.numRegs * 32 + 255) / 256) * 256;  // allocated per warp in units of 256
    int n = 512 / (int)kTmemCols;
    const int by_smem = (int)(smem_sm / (smem + fa.sharedSizeBytes + (size_t)reserved));
    const int by_regs = regs_sm / (regs_warp * (kThreads / 32));
    n = n < by_smem ? n : by_smem;
    n = n < by_regs ? n : by_regs;
    if (n < 1) return cudaErrorInvalidConfiguration;
    if (dev < 64) cached[dev][split] = n;
    *per_sm = n;
    return cudaSuccess;
}

cudaError_t beams_plan(int N, int K, int Hq, int Hkv, int max_pages, int num_workers, BeamsPlan* plan) {
    const size_t R = (size_t)K * (Hq / Hkv);
    int per_sm = 0, sms = 0;
    const cudaError_t e = beams_occupancy((int)R, &per_sm, &sms);
    if (e != cudaSuccess) return e;
    auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
    plan->tc_grid = num_workers > 0 ? num_workers : (long long)sms * per_sm;
    plan->slots = (size_t)plan->tc_grid + (size_t)N * Hkv;  // partial slot = share + segment
    plan->part_lse_offset = up(plan->slots * R * kHeadDim * 4);
    plan->merge_list_offset = up(plan->part_lse_offset + plan->slots * R * 4);
    plan->counts_offset = up(plan->merge_list_offset + (size_t)plan->tc_grid * sizeof(int2));
    plan->entries_offset = up(plan->counts_offset + (size_t)N * 4);
    plan->ws_bytes = plan->entries_offset + (size_t)N * K * max_pages * sizeof(PageEntry);
    return cudaSuccess;
}

cudaError_t decode_beams_launch(const BeamsArgs& args, const CUtensorMap& tq, const CUtensorMap& tk,
                                const CUtensorMap& tv, bool may_split, cudaStream_t stream) {
    if (args.N == 0) return cudaSuccess;
    if (args.tc_grid > 0x7fffffffll || args.tc_grid < 1) return cudaErrorInvalidConfiguration;
    int per_sm = 0, sms = 0, split = 1;  // the call also sets the kernel's shared-memory limit
    cudaError_t e = beams_occupancy(args.R, &per_sm, &sms);
    if (e != cudaSuccess) return e;
    BeamsArgs a = args;
    if (!may_split) a.merge_list = nullptr;
    // the plan: as many lanes a column as rows, two columns a lane where a CTA's threads are enough, else up to
    // kPlanSteps; clusters of up to eight CTAs, while all groups' CTAs find room on half of the SMs or the columns need them
    const int lanes = a.K <= 4 ? 4 : (a.K <= 8 ? 8 : (a.K <= 16 ? 16 : 32));
    const long long wanted = (long long)a.max_pages * lanes;
    int ctas = 1;
    while (ctas < 8 && wanted > 2048ll * ctas && ((long long)a.N * ctas * 4 <= sms || wanted > 1024ll * kPlanSteps * ctas)) ctas *= 2;
    const long long half = (wanted / ctas + 1) / 2, warps = (half + 31) / 32;
    const int threads = warps >= 32 ? 1024 : (int)warps * 32;
    const long long rounds = (wanted + (long long)ctas * threads - 1) / ((long long)ctas * threads);
    const int steps = rounds < kPlanSteps ? (int)rounds : kPlanSteps;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.N * ctas));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = lanes == 4    ? cudaLaunchKernelEx(&cfg, beams_plan_kernel<4>, a, steps)
        : lanes == 8  ? cudaLaunchKernelEx(&cfg, beams_plan_kernel<8>, a, steps)
        : lanes == 16 ? cudaLaunchKernelEx(&cfg, beams_plan_kernel<16>, a, steps)
                      : cudaLaunchKernelEx(&cfg, beams_plan_kernel<32>, a, steps);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)a.tc_grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = 1024 + sizeof(Smem);
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, beams_kernel(a.R, &split), tq, tk, tv, a);
    if (e != cudaSuccess || !may_split) return e;
    SplitMergeArgs m;
    m.part_o = a.part_o;
    m.part_lse = a.part_lse;
    m.list = a.merge_list;
    m.out = a.out;
    m.lse = a.lse;
    m.listed = (int)a.tc_grid;
    m.R = a.R;
    m.G = a.G;
    m.QL = a.K;
    m.Hq = a.Hq;
    m.Hkv = a.Hkv;
    return split_merge_launch(m, stream);
}

}  // namespace sinkattn
