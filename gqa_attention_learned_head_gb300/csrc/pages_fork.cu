// pages_fork.cu -- page tables, page counts and page copies of one step that forks, drops, trims and grows
// rows of a paged cache.
//
// Whole numbers only.  With kc = ceil(keep / 16), rc = ceil(room / 16), hc = ceil(held / 16) columns, row r
// takes columns [0, kc) from its parent, and rc - kc new pages (one more where its last kept page is replaced,
// see replaces below).  The pages' counts change by
//   +1 for every kept column of every child but a parent's first,
//   -1 for every column that a parent holds beyond those its first child keeps (all of them without a child),
// which is the sum over all rows with the first child's and its parent's +1 and -1 left out: a row that simply
// goes on touches no count.  New pages count 1.  Additions commute, so no order shows in the result.
//
// fork_plan_kernel: one cluster of CTAs.  First, least and greatest keep of every parent's children (atomic
// minimum and maximum), a prefix sum over the rows' needs, and the lowest free pages from one pass over the counts
// (which also copies them): a bit for every page of the pass stays in registers until the sums of the cluster
// (through distributed shared memory) have said where each thread's free pages go.  Its time is latency: chains of
// loads (a row's parent, its parent's tokens, its last page, that page's count) and barriers.  So up to kLocalRows
// rows every CTA goes over all of them by itself, in shared memory, and the cluster meets once.
// fork_apply_kernel: a thread takes a column or some of kBatch present and kBatch new rows, reads and writes their
// entries, and adds up the changes to the count of a page that several of them hold: for the pages that a group's
// rows share, drops and forks mostly cancel and no atomic is left.  Its loads are latency too: a group's rows are read
// together, and a quarter of the time is the table's bytes.
//
// Measured (GB300): 256 groups of 8 rows of 1024 to 32768 tokens (27.8 MB: 4.1 us at the copy rate) 24.0 us, 12.5 in the
// plan and 11.5 in the application; 4 rows of one group 7.5 us; 1024 groups of 8, over kLocalRows, 55.7 us (111 MB: 16.4 us).
// The simplest form
// (an atomic for every holder that comes or goes) took 54 us.
#include "args_pages.h"
#include "errors_beam.h"
#include "ptx.cuh"

#include <climits>
#include <cooperative_groups.h>

namespace cg = cooperative_groups;

namespace sinkattn {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPass = 32 * kPlanThreads;  // pages that a CTA takes in one pass, a word of 32 a thread
constexpr int kWords = 2;                 // passes whose words a thread keeps
constexpr int kLocalRows = 4096;          // rows that every CTA of the plan goes over itself
constexpr int kApplyThreads = 128;
// rows of a thread of the apply kernel: with 256 groups of 8 rows of 1024 to 32768 tokens the call takes 24.0 us with 4,
// 28.2 with 8 (more registers, fewer threads) and 27.1 with 2 (fewer changes cancel)
constexpr int kBatch = 4;
constexpr unsigned kTop = 0x80000000u;

__device__ __forceinline__ int cols(int tokens) { return (tokens + kPageSize - 1) / kPageSize; }

// A new row's parent, kept and room tokens, brought into range, and the count of the page that it is going to
// write: kNoPage if it writes none, or one that is not of the pool.
constexpr int kNoPage = INT_MIN;
struct Row {
    int parent, keep, room, count;
    __device__ bool writes() const { return room > keep && keep % kPageSize != 0; }  // its last kept page
};
// Rows r .. r + n - 1 (n <= N), the loads of each kind issued together; `bad` collects the error bits.
template <int N>
__device__ __forceinline__ void load_rows(const ForkArgs& a, int r, int n, Row (&x)[N], unsigned& bad) {
    const int cap = a.max_pages * kPageSize;
    int keep[N], room[N], held[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        x[i] = Row{-1, 0, 0, kNoPage};
        keep[i] = room[i] = 0;
        if (i < n) {
            x[i].parent = __ldcg(&a.parents[r + i]);
            if (a.keep_lens) keep[i] = __ldcg(&a.keep_lens[r + i]);
            if (a.room_lens) room[i] = __ldcg(&a.room_lens[r + i]);
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (x[i].parent < -1 || x[i].parent >= a.Rin) {
            bad |= kErrBadIndex;
            x[i].parent = -1;
        }
        held[i] = x[i].parent >= 0 ? __ldcg(&a.held_lens[x[i].parent]) : 0;
    }
    int page[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int h = held[i] < 0 ? 0 : (held[i] > cap ? cap : held[i]);  // reported where the parent is looked at
        x[i].keep = h;
        if (a.keep_lens) {
            if (keep[i] < 0 || keep[i] > h) bad |= kErrBadLength;
            x[i].keep = keep[i] < 0 ? 0 : (keep[i] > h ? h : keep[i]);
        }
        long long m = x[i].parent >= 0 ? (long long)x[i].keep + a.grow : 0;
        if (a.room_lens) m = room[i];
        if (m < x[i].keep || m > cap) {
            if (i < n) bad |= kErrBadLength;
            m = m < x[i].keep ? x[i].keep : cap;
        }
        x[i].room = i < n ? (int)m : 0;
        page[i] = x[i].writes() ? __ldcg(&a.page_table[(long long)x[i].parent * a.max_pages + x[i].keep / kPageSize]) : -1;
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (page[i] >= 0 && page[i] < a.P) x[i].count = __ldcg(&a.refs_in[page[i]]);
}
// Whether row r gets a new page in place of its last kept one: it will write that page (a page of the pool), and is
// not the first of children that all keep the same and will write, of the page's one holder.
__device__ __forceinline__ bool replaces(int r, int count, int first, int low, int high) {
    return count != kNoPage && !(count == 1 && first == r && low == high);
}

// Inclusive prefix sum over the CTA's threads; `total` is the sum.  red: one word per warp.
__device__ __forceinline__ long long block_scan(long long v, long long* red, long long& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    __syncthreads();
    if (lane == 31) red[warp] = v;
    __syncthreads();
    long long w = red[lane];
    const long long own = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    total = __shfl_sync(0xffffffffu, w, 31);
    return v + __shfl_sync(0xffffffffu, w - own, warp);
}

// Free pages among p .. p + 1023 (below `end`), p the warp's first: lane l's word has bit i set where page
// p + 32 l + i is free.  Sixteen bytes a lane and step, eight steps in flight; a step's eight neighbouring lanes make a word.
__device__ __forceinline__ unsigned free_word(const int* counts, bool wide, long long p, int end) {
    const int lane = threadIdx.x & 31;
    if (p >= end) return 0u;
    int4 c[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const long long q = p + 128 * j + 4 * lane;
        if (wide && q + 4 <= end) {
            c[j] = __ldcg(reinterpret_cast<const int4*>(counts + q));
        } else {
            c[j].x = q < end ? __ldcg(counts + q) : -1;
            c[j].y = q + 1 < end ? __ldcg(counts + q + 1) : -1;
            c[j].z = q + 2 < end ? __ldcg(counts + q + 2) : -1;
            c[j].w = q + 3 < end ? __ldcg(counts + q + 3) : -1;
        }
    }
    unsigned mine = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        unsigned w = ((c[j].x == 0) | (c[j].y == 0) << 1 | (c[j].z == 0) << 2 | (c[j].w == 0) << 3) << (4 * (lane & 7));
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) w |= __shfl_xor_sync(0xffffffffu, w, o);
        mine = (lane & 7) == j ? w : mine;  // lane 8 g + j has word 4 j + g
    }
    return __shfl_sync(0xffffffffu, mine, 8 * (lane & 3) + (lane >> 2));
}

struct PlanSmem {
    long long red[kPlanThreads / 32];
    long long sums[2];  // this CTA's new pages needed, free pages found
    int first[kLocalRows], low[kLocalRows], high[kLocalRows], keep[kLocalRows];  // LOCAL
};

// The first cluster plans, any further ones copy the counts.
// LOCAL: every CTA of the cluster goes over all the rows, at most kLocalRows present and new ones, with the parents'
// children in its own shared memory; else each over its part of the rows, with the children in the workspace.
template <bool LOCAL>
__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const ForkArgs a) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    PlanSmem& sm = *reinterpret_cast<PlanSmem*>(smem_raw);
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
    const bool wide = ((reinterpret_cast<uintptr_t>(a.refs_in) | reinterpret_cast<uintptr_t>(a.refs_out)) & 15) == 0;
    if ((int)blockIdx.x >= ctas) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        const long long first = (long long)((int)blockIdx.x - ctas) * kPlanThreads + tid;
        const long long step = (long long)((int)gridDim.x - ctas) * kPlanThreads, quads = wide ? a.P / 4 : 0;
        for (long long i = first; i < quads; i += step)
            reinterpret_cast<int4*>(a.refs_out)[i] = __ldcg(reinterpret_cast<const int4*>(a.refs_in) + i);
        for (long long i = 4 * quads + first; i < a.P; i += step) a.refs_out[i] = __ldcg(&a.refs_in[i]);
        return;
    }
    int* first = LOCAL ? sm.first : a.first;
    int* low = LOCAL ? sm.low : a.low;
    int* high = LOCAL ? sm.high : a.high;
    // the pages of this CTA, and the rows that it goes over, a run of `per` consecutive ones a thread; the last threads
    // take the first rows, as the first take the first pages: with little to do, both run at once
    const long long p_len = (((long long)a.P + ctas - 1) / ctas + 3) & ~3ll;
    const int p0 = (int)min((long long)a.P, rank * p_len), p1 = (int)min((long long)a.P, p0 + p_len);
    const int r_len = LOCAL ? a.Rout : (a.Rout + ctas - 1) / ctas, turned = kPlanThreads - 1 - tid;
    const int r0 = LOCAL ? 0 : min(a.Rout, rank * r_len), r1 = min(a.Rout, r0 + r_len);
    const int per = (r1 - r0 + kPlanThreads - 1) / kPlanThreads;
    const int ra = (int)min((long long)r1, r0 + (long long)turned * per), rb = min(r1, ra + per);
    const int stride = LOCAL ? kPlanThreads : kPlanThreads * ctas, start = LOCAL ? tid : rank * kPlanThreads + tid;
    const bool report = !LOCAL || rank == 0;
    unsigned bad = 0;
    if constexpr (LOCAL)
        for (int p = start; p < a.Rin; p += stride) {
            first[p] = INT_MAX;
            low[p] = INT_MAX;
            high[p] = INT_MIN;
        }
    if (tid == 0) sm.sums[1] = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- 1. the rows (LOCAL: a thread's stay in registers), and the pass over the counts
    constexpr int kHeld = LOCAL ? kLocalRows / kPlanThreads : 1;
    Row held[kHeld];
    if (ra < rb) load_rows(a, ra, min(kHeld, rb - ra), held, bad);
    auto row = [&](int r, unsigned& seen) {
        if constexpr (LOCAL) {
            Row x = held[0];
#pragma unroll
            for (int i = 1; i < kHeld; ++i) x = r == ra + i ? held[i] : x;
            return x;
        } else {
            if (r == ra) return held[0];
            Row x[1];
            load_rows(a, r, 1, x, seen);
            return x[0];
        }
    };
    if constexpr (!LOCAL)
        for (int p = start; p < a.Rin; p += stride) {
            first[p] = INT_MAX;
            low[p] = INT_MAX;
            high[p] = INT_MIN;
        }
    unsigned words[kWords];
    int found = 0;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
        words[i] = free_word(a.refs_in, wide, (long long)p0 + (long long)i * kPass + 1024 * warp, p1);
        found += __popc(words[i]);
    }
    for (long long q = (long long)p0 + kWords * kPass; q < p1; q += kPass)  // read again below
        found += __popc(free_word(a.refs_in, wide, q + 1024 * warp, p1));
    found = __reduce_add_sync(0xffffffffu, found);
    if constexpr (LOCAL) __syncthreads();
    else cluster.sync();

    // ---- 2. each parent's children
    if (lane == 0 && found) atomicAdd(reinterpret_cast<unsigned long long*>(&sm.sums[1]), (unsigned long long)found);
    for (int r = ra; r < rb; ++r) {
        const Row x = row(r, bad);
        if constexpr (LOCAL) sm.keep[r] = x.keep;
        if (x.parent < 0) continue;
        const int mark = x.writes() ? x.keep : -1;
        atomicMin(&first[x.parent], r);
        atomicMin(&low[x.parent], mark);
        atomicMax(&high[x.parent], mark);
    }
    if constexpr (LOCAL) __syncthreads();
    else cluster.sync();

    // ---- 3. the rows' needs and their prefix; the sums of the cluster
    auto need_of = [&](int r, Row& x, bool& replace, bool& is_first) {
        unsigned ignored = 0;
        x = row(r, ignored);
        replace = is_first = false;
        if (x.parent >= 0) {
            const int f = LOCAL ? first[x.parent] : __ldcg(&first[x.parent]);
            const int lo = LOCAL ? low[x.parent] : __ldcg(&low[x.parent]), hi = LOCAL ? high[x.parent] : __ldcg(&high[x.parent]);
            is_first = f == r;
            replace = replaces(r, x.count, f, lo, hi);
        }
        return cols(x.room) - cols(x.keep) + (int)replace;
    };
    Row x;
    bool replace, is_first;
    long long need = 0, need_all;
    for (int r = ra; r < rb; ++r) need += need_of(r, x, replace, is_first);
    // (the threads' prefix runs over the rows from behind)
    long long at = block_scan(need, sm.red, need_all);
    at = need_all - at;
    if (tid == 0) sm.sums[0] = need_all;
    cluster.sync();
    long long free_before = 0, free_all = 0, need_sum = 0;
    for (int i = 0; i < ctas; ++i) {
        const long long* s = cluster.map_shared_rank(sm.sums, i);
        const long long n = s[0], f = s[1];
        if (!LOCAL) at += i < rank ? n : 0;
        free_before += i < rank ? f : 0;
        need_sum += n;
        free_all += f;
    }
    if (!LOCAL) need_all = need_sum;
    auto leave = cluster.barrier_arrive();  // no CTA ends while another reads its sums
    const bool ok = need_all <= free_all;
    if (rank == 0 && tid == 0) {
        *a.ok = ok ? 1 : 0;
        if (!ok) atomicOr(a.err, kErrNoPages);
    }

    // ---- 4. the records of the new and of the present rows (LOCAL: the first CTA's), and the lowest free pages in order
    if (report) {
        for (int r = ra; r < rb; ++r) {
            const int n = need_of(r, x, replace, is_first);
            const unsigned from = (unsigned)min((long long)INT_MAX, at) | (replace ? kTop : 0u);
            a.rows[r] = make_int4(x.parent, x.keep, (int)((unsigned)x.room | (is_first ? kTop : 0u)), (int)from);
            at += n;
        }
        for (int p = start; p < a.Rin; p += stride) {
            const int h = __ldcg(&a.held_lens[p]), cap = a.max_pages * kPageSize;
            if (h < 0 || h > cap) bad |= kErrBadLength;
            const int f = LOCAL ? first[p] : __ldcg(&first[p]);
            int kept = 0;
            if (f != INT_MAX) {
                if constexpr (LOCAL) {
                    kept = sm.keep[f];
                } else {
                    unsigned ignored = 0;
                    Row y[1];
                    load_rows(a, f, 1, y, ignored);
                    kept = y[0].keep;
                }
            }
            a.drops[p] = make_int2(cols(kept), cols(h < 0 ? 0 : (h > cap ? cap : h)));
        }
        if (bad) atomicOr(a.err, bad);
    }
    if (ok) {
        int pass = 0;
        for (long long q = p0; q < p1 && free_before < need_all; q += kPass, ++pass) {
            const long long mine = q + 1024 * warp;
            unsigned w = pass < kWords ? words[0] : free_word(a.refs_in, wide, mine, p1);
#pragma unroll
            for (int i = 1; i < kWords; ++i) w = pass == i ? words[i] : w;
            long long total, spot = free_before + block_scan(__popc(w), sm.red, total) - __popc(w);
            for (; w && spot < need_all; w &= w - 1) a.free_ids[spot++] = (int)(mine + 32 * lane) + __ffs(w) - 1;
            free_before += total;
        }
    }
    cluster.barrier_wait(std::move(leave));
}

template <int VEC>
struct Pages {
    int v[VEC];
};
template <int VEC>
__device__ __forceinline__ Pages<VEC> load_pages(const int* p) {
    Pages<VEC> x;
    if constexpr (VEC == 4) {
        const int4 y = __ldcg(reinterpret_cast<const int4*>(p));
        x.v[0] = y.x;
        x.v[1] = y.y;
        x.v[2] = y.z;
        x.v[3] = y.w;
    } else if constexpr (VEC == 2) {
        const int2 y = __ldcg(reinterpret_cast<const int2*>(p));
        x.v[0] = y.x;
        x.v[1] = y.y;
    } else {
        x.v[0] = __ldcg(p);
    }
    return x;
}
template <int VEC>
__device__ __forceinline__ void store_pages(int* p, const Pages<VEC>& x) {
    if constexpr (VEC == 4) *reinterpret_cast<int4*>(p) = make_int4(x.v[0], x.v[1], x.v[2], x.v[3]);
    else if constexpr (VEC == 2) *reinterpret_cast<int2*>(p) = make_int2(x.v[0], x.v[1]);
    else *p = x.v[0];
}

// A new row as the apply kernel uses it: columns [0, kept) from its parent's row, [kept, rc) new pages.
struct ApplyRow {
    const int* from;   // its parent's row
    const int* fresh;  // fresh[c] is column c's new page
    int kept, rc;
};
// The pages of columns [begin, end) of a row lose or gain a holder.
struct Change {
    const int* row;
    int begin, end, by;
};

// Block b of `chunks` blocks a batch: columns kApplyThreads VEC (b % chunks) on, VEC a thread, of present and of new rows
// kBatch (b / chunks) on.  The counts are only added to here (they may be the call's input): what depends on them was
// decided by the plan.
template <int VEC>
__global__ void __launch_bounds__(kApplyThreads) fork_apply_kernel(const ForkArgs a, const int chunks) {
    __shared__ ApplyRow rows[kBatch];
    __shared__ Change changes[2 * kBatch];
    __shared__ int num_changes;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, batch = (int)(blockIdx.x / (unsigned)chunks), chunk = (int)(blockIdx.x % (unsigned)chunks);
    // the block's columns [lo, hi) (as if whole) and the thread's first
    const int b0 = batch * kBatch, lo = chunk * kApplyThreads * VEC, hi = lo + kApplyThreads * VEC, c0 = lo + tid * VEC;
    const int n_out = min(kBatch, a.Rout - b0), n_in = min(kBatch, a.Rin - b0);  // may be negative
    const bool ok = __ldcg(a.ok) != 0;
    int4 mine = make_int4(-1, 0, 0, 0);
    ApplyRow x = {nullptr, nullptr, 0, 0};
    if (tid < 32) {
        // lanes 0 .. kBatch - 1 the new rows, the next ones the present rows; the changes that touch this block, losses first
        Change y = {nullptr, 0, 0, 0};
        const int i = tid - kBatch;
        if (tid < n_out) {
            mine = __ldcg(&a.rows[b0 + tid]);
            x.kept = cols(mine.y) - (int)((unsigned)mine.w >> 31);
            x.rc = cols(mine.z & 0x7fffffff);
            x.from = a.page_table + (long long)mine.x * a.max_pages;
            x.fresh = a.free_ids + (mine.w & 0x7fffffff) - x.kept;
            rows[tid] = x;
            if (mine.z >= 0) y = Change{x.from, 0, x.kept, 1};  // not its parent's first child
        } else if (i >= 0 && i < n_in) {
            const int2 d = __ldcg(&a.drops[b0 + i]);
            y = Change{a.page_table + (long long)(b0 + i) * a.max_pages, d.x, d.y, -1};
        }
        const bool here = y.end > lo && y.begin < hi && y.end > y.begin;
        const unsigned below = (1u << tid) - 1, gains = __ballot_sync(0xffffffffu, here && y.by > 0),
                       losses = __ballot_sync(0xffffffffu, here && y.by < 0);
        if (here) changes[y.by < 0 ? __popc(losses & below) : __popc(losses) + __popc(gains & below)] = y;
        if (tid == 0) num_changes = __popc(losses | gains);
    }
    __syncthreads();
    Pages<VEC> none;
#pragma unroll
    for (int v = 0; v < VEC; ++v) none.v[v] = -1;
    if (!ok) {
        for (int i = 0; i < n_out; ++i) {
            const long long r = b0 + i;
            if (c0 < a.max_pages) store_pages<VEC>(&a.out_table[r * a.max_pages + c0], none);
            if (chunk == 0 && tid == 0) a.out_lens[r] = 0;
            if (chunk == 0 && tid < 3) a.copies[3 * r + tid] = tid < 2 ? -1 : 0;
        }
        return;
    }
    bool bad = false;
    if (c0 < a.max_pages) {
        // ---- the new rows' entries
        Pages<VEC> now[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            now[i] = none;
            if (i < n_out && c0 < rows[i].kept) now[i] = load_pages<VEC>(rows[i].from + c0);
        }
        // ---- the first changes' pages, on their way meanwhile
        const int n = num_changes;
        Pages<VEC> at[kBatch];
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
            at[e] = none;
            if (e < n && c0 < changes[e].end) at[e] = load_pages<VEC>(changes[e].row + c0);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (i >= n_out) break;
            if (hi > rows[i].kept) {  // new pages, or nothing, in some of the block's columns
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    const int c = c0 + v;
                    if (c < rows[i].kept) {
                        bad |= (unsigned)now[i].v[v] >= (unsigned)a.P;
                    } else if (c < rows[i].rc) {
                        now[i].v[v] = __ldcg(rows[i].fresh + c);
                        a.refs_out[now[i].v[v]] = 1;  // free until now: nothing else adds to it
                    } else {
                        now[i].v[v] = -1;
                    }
                }
            } else {
#pragma unroll
                for (int v = 0; v < VEC; ++v) bad |= (unsigned)now[i].v[v] >= (unsigned)a.P;
            }
            store_pages<VEC>(&a.out_table[(long long)(b0 + i) * a.max_pages + c0], now[i]);
        }
        // ---- the changes of a column, one after another, added up while they are of the same page
        int page[VEC], sum[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) page[v] = sum[v] = 0;
        auto flush = [&](int v) {
            if (sum[v]) atomicAdd(&a.refs_out[page[v]], sum[v]);
            sum[v] = 0;
        };
        auto add = [&](const Change& y, const Pages<VEC>& p) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                if (c0 + v < y.begin || c0 + v >= y.end) continue;
                if ((unsigned)p.v[v] >= (unsigned)a.P) {
                    bad = true;
                    continue;
                }
                if (p.v[v] != page[v]) {
                    flush(v);
                    page[v] = p.v[v];
                }
                sum[v] += y.by;
            }
        };
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
            if (e >= n) break;
            add(changes[e], at[e]);
        }
#pragma unroll 1
        for (int e = kBatch; e < n; ++e)
            if (c0 < changes[e].end) add(changes[e], load_pages<VEC>(changes[e].row + c0));
#pragma unroll
        for (int v = 0; v < VEC; ++v) flush(v);
    }
    if (chunk == 0 && tid < n_out) {
        const bool replace = mine.w < 0;
        int src = -1, dst = -1, tokens = 0;
        if (replace) {
            src = __ldcg(x.from + x.kept);
            dst = __ldcg(x.fresh + x.kept);
            tokens = mine.y % kPageSize;
            if (mine.z < 0) atomicSub(&a.refs_out[src], 1);  // the first child does not go on in its parent's page
        }
        const long long r = b0 + tid;
        a.out_lens[r] = mine.z & 0x7fffffff;
        a.copies[3 * r] = src;
        a.copies[3 * r + 1] = dst;
        a.copies[3 * r + 2] = tokens;
    }
    if (bad) atomicOr(a.err, kErrBadPage);
}

// The plan's shared memory, allowed once per device and thread.
cudaError_t allow_smem(const void* kernel, bool local, size_t bytes) {
    static thread_local bool allowed[64][2] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && allowed[dev][local])) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess && dev < 64) allowed[dev][local] = true;
    return e;
}

}  // namespace

void fork_plan(int Rin, int Rout, int P, ForkPlan* plan) {
    auto up = [](size_t x) { return (x + 15) & ~size_t(15); };
    plan->drops = up(size_t(Rout) * sizeof(int4));
    plan->first = up(plan->drops + size_t(Rin) * sizeof(int2));
    plan->low = up(plan->first + size_t(Rin) * 4);
    plan->high = up(plan->low + size_t(Rin) * 4);
    plan->free_ids = up(plan->high + size_t(Rin) * 4);
    plan->ok = up(plan->free_ids + size_t(P) * 4);
    plan->ws_bytes = plan->ok + 4;
}

cudaError_t pages_fork_launch(const ForkArgs& a, cudaStream_t stream) {
    // one CTA while a row or a step of pages per thread are all there is, else a cluster of eight
    const int ctas = a.Rin <= kPlanThreads && a.Rout <= kPlanThreads && a.P <= 4 * kPlanThreads ? 1 : 8;
    const bool local = a.Rin <= kLocalRows && a.Rout <= kLocalRows;
    void (*plan)(const ForkArgs) = local ? fork_plan_kernel<true> : fork_plan_kernel<false>;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(plan), local, sizeof(PlanSmem));
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    // behind the planning cluster, clusters that copy the counts, four steps of a thread each
    const int copiers = a.refs_out == a.refs_in ? 0 : (a.P / (16 * kPlanThreads * ctas) < 16 ? a.P / (16 * kPlanThreads * ctas) + 1 : 16);
    cfg.gridDim = dim3((unsigned)(ctas * (1 + copiers)));
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = sizeof(PlanSmem);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if ((e = cudaLaunchKernelEx(&cfg, plan, a)) != cudaSuccess) return e;
    cfg.dynamicSmemBytes = 0;
    const int rows = a.Rin > a.Rout ? a.Rin : a.Rout;
    if (rows == 0) return cudaSuccess;
    // as many columns a thread as every row of both tables allows loads of
    const bool even = ((reinterpret_cast<uintptr_t>(a.page_table) | reinterpret_cast<uintptr_t>(a.out_table)) & 15) == 0;
    const int vec = !even ? 1 : (a.max_pages % 4 == 0 ? 4 : (a.max_pages % 2 == 0 ? 2 : 1));
    const int chunks = (a.max_pages + kApplyThreads * vec - 1) / (kApplyThreads * vec);
    const long long blocks = (long long)((rows + kBatch - 1) / kBatch) * chunks;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kApplyThreads);
    cfg.numAttrs = 1;
    return vec == 4   ? cudaLaunchKernelEx(&cfg, fork_apply_kernel<4>, a, chunks)
           : vec == 2 ? cudaLaunchKernelEx(&cfg, fork_apply_kernel<2>, a, chunks)
                      : cudaLaunchKernelEx(&cfg, fork_apply_kernel<1>, a, chunks);
}

}  // namespace sinkattn
