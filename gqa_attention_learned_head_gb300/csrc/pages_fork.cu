// pages_fork.cu -- page tables, page counts and page copies of one step that forks, drops, trims and grows
// rows of a paged cache.
//
// Whole numbers only.  With kc = ceil(keep / 16), rc = ceil(room / 16), hc = ceil(held / 16) columns, row r
// takes columns [0, kc) from its parent, and rc - kc new pages (one more where its last kept page is replaced,
// see row_of below).  The pages' counts change by
//   +1 for every kept column of every child but a parent's first,
//   -1 for every column that a parent holds beyond those its first child keeps (all of them without a child),
// which is the sum over all rows with the first child's and its parent's +1 and -1 left out: a row that simply
// goes on touches no count.  New pages count 1.  Additions commute, so no order shows in the result.
//
// fork_plan_kernel: one cluster of CTAs.  First, least and greatest keep of every parent's children (atomic
// minimum and maximum), a prefix sum over the rows' needs and, in the same pass as the copy of the counts, the
// lowest free pages, both by cluster-wide scans through distributed shared memory.  Its time is latency (three
// cluster barriers around passes over a few MB in L2).  fork_apply_kernel: one CTA per row (new rows write
// their table, present rows give up their columns), bound by the table's bytes and the counts' atomics.
#include "args_pages.h"
#include "ptx.cuh"

#include <climits>
#include <cooperative_groups.h>

namespace cg = cooperative_groups;

namespace sinkattn {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kApplyThreads = 128;

__device__ __forceinline__ int cols(int tokens) { return (tokens + kPageSize - 1) / kPageSize; }

// A present row's held tokens, clamped.
__device__ __forceinline__ int held_of(const ForkArgs& a, int p) {
    const int h = __ldcg(&a.held_lens[p]), cap = a.max_pages * kPageSize;
    return h < 0 ? 0 : (h > cap ? cap : h);
}

// A new row's parent, kept and room tokens, brought into range; `bad` collects the error bits.
struct Row {
    int parent, keep, room;
    bool writes;  // its last kept page is partial and will be written
};
__device__ __forceinline__ Row row_of(const ForkArgs& a, int r, unsigned& bad) {
    const int cap = a.max_pages * kPageSize;
    Row x;
    x.parent = __ldcg(&a.parents[r]);
    if (x.parent < -1 || x.parent >= a.Rin) {
        bad |= kErrBadIndex;
        x.parent = -1;
    }
    const int held = x.parent >= 0 ? held_of(a, x.parent) : 0;
    x.keep = held;
    if (a.keep_lens) {
        x.keep = __ldcg(&a.keep_lens[r]);
        if (x.keep < 0 || x.keep > held) {
            bad |= kErrBadLength;
            x.keep = x.keep < 0 ? 0 : held;
        }
    }
    long long room = x.parent >= 0 ? (long long)x.keep + a.grow : 0;
    if (a.room_lens) room = __ldcg(&a.room_lens[r]);
    if (room < x.keep || room > cap) {
        bad |= kErrBadLength;
        room = room < x.keep ? x.keep : cap;
    }
    x.room = (int)room;
    x.writes = x.room > x.keep && x.keep % kPageSize != 0;
    return x;
}

// Whether row r gets a new page in place of its last kept one.
__device__ __forceinline__ bool replaces(const ForkArgs& a, int r, const Row& x, int first, int low, int high) {
    if (!x.writes) return false;
    const int page = __ldcg(&a.page_table[(long long)x.parent * a.max_pages + x.keep / kPageSize]);
    if (page < 0 || page >= a.P) return false;  // not a page of the pool: carried along
    return !(__ldcg(&a.refs_in[page]) == 1 && first == r && low == high);
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
    long long w = lane < kPlanThreads / 32 ? red[lane] : 0;
    const long long own = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    total = __shfl_sync(0xffffffffu, w, 31);
    return v + __shfl_sync(0xffffffffu, w - own, warp);
}

__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const ForkArgs a) {
    __shared__ long long red[kPlanThreads / 32];
    __shared__ long long sums[2];  // this CTA's new pages needed, free pages found
    cg::cluster_group cluster = cg::this_cluster();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
    const int gt = rank * kPlanThreads + tid, gn = ctas * kPlanThreads;
    unsigned bad = 0;

    // ---- 1. each parent's children
    for (int p = gt; p < a.Rin; p += gn) {
        a.first[p] = INT_MAX;
        a.low[p] = INT_MAX;
        a.high[p] = INT_MIN;
        const int h = __ldcg(&a.held_lens[p]);
        if (h < 0 || h > a.max_pages * kPageSize) bad |= kErrBadLength;
    }
    cluster.sync();
    for (int r = gt; r < a.Rout; r += gn) {
        const Row x = row_of(a, r, bad);
        if (x.parent < 0) continue;
        const int mark = x.writes ? x.keep : -1;
        atomicMin(&a.first[x.parent], r);
        atomicMin(&a.low[x.parent], mark);
        atomicMax(&a.high[x.parent], mark);
    }
    if (bad) atomicOr(a.err, bad);
    cluster.sync();

    // ---- 2. the rows' needs and the free pages, counted; each CTA a contiguous part of both
    const int r_len = (a.Rout + ctas - 1) / ctas, r0 = min(a.Rout, rank * r_len), r1 = min(a.Rout, r0 + r_len);
    const int p_len = ((a.P + ctas - 1) / ctas + 3) & ~3, p0 = min(a.P, rank * p_len), p1 = min(a.P, p0 + p_len);
    auto need_of = [&](int r, bool& replace) {
        unsigned ignored = 0;
        const Row x = row_of(a, r, ignored);
        replace = x.parent >= 0 && replaces(a, r, x, __ldcg(&a.first[x.parent]), __ldcg(&a.low[x.parent]),
                                            __ldcg(&a.high[x.parent]));
        return cols(x.room) - cols(x.keep) + (int)replace;
    };
    long long need = 0, free = 0, total;
    bool replace = false;
    for (int r = r0 + tid; r < r1; r += kPlanThreads) need += need_of(r, replace);
    for (int p = p0 + tid; p < p1; p += kPlanThreads) {
        const int c = __ldcg(&a.refs_in[p]);
        free += c == 0;
    }
    block_scan(need, red, total);
    if (tid == 0) sums[0] = total;
    block_scan(free, red, total);
    if (tid == 0) sums[1] = total;
    cluster.sync();
    long long need_before = 0, need_all = 0, free_before = 0, free_all = 0;
    for (int i = 0; i < ctas; ++i) {
        const long long* s = cluster.map_shared_rank(sums, i);
        need_before += i < rank ? s[0] : 0;
        free_before += i < rank ? s[1] : 0;
        need_all += s[0];
        free_all += s[1];
    }
    cluster.sync();  // no CTA ends while another reads its sums
    const bool ok = need_all <= free_all;
    if (rank == 0 && tid == 0) {
        *a.ok = ok ? 1 : 0;
        if (!ok) atomicOr(a.err, kErrNoPages);
    }

    // ---- 3. where each row's new pages start, and the lowest free pages in order; the counts are copied
    for (int base = r0; base < r1; base += kPlanThreads) {
        const int r = base + tid;
        const int n = r < r1 ? need_of(r, replace) : 0;
        const long long incl = block_scan(n, red, total);
        if (r < r1) a.at[r] = (int)((unsigned)min((long long)INT_MAX, need_before + incl - n) | (replace ? 1u << 31 : 0u));
        need_before += total;
    }
    const bool copy = a.refs_out != a.refs_in;
    for (int base = p0; base < p1; base += kPlanThreads) {
        const int p = base + tid;
        int is_free = 0;
        if (p < p1) {
            const int c = __ldcg(&a.refs_in[p]);
            is_free = c == 0;
            if (copy) a.refs_out[p] = c;
        }
        const long long incl = block_scan(is_free, red, total);
        const long long spot = free_before + incl - 1;
        if (is_free && ok && spot < need_all) a.free_ids[spot] = p;
        free_before += total;
    }
}

// Blocks [0, Rout) write the new rows, blocks [Rout, Rout + Rin) give up what the present rows held.  The counts
// are only added to here (they may be the call's input): what depends on them was decided by the plan.
__global__ void __launch_bounds__(kApplyThreads) fork_apply_kernel(const ForkArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x;
    const bool ok = __ldcg(a.ok) != 0;
    unsigned bad = 0, ignored = 0;
    if ((int)blockIdx.x < a.Rout) {
        const int r = (int)blockIdx.x;
        int* out = a.out_table + (long long)r * a.max_pages;
        if (!ok) {
            for (int c = tid; c < a.max_pages; c += kApplyThreads) out[c] = -1;
            if (tid == 0) a.out_lens[r] = 0;
            if (tid < 3) a.copies[3ll * r + tid] = tid < 2 ? -1 : 0;
            return;
        }
        const Row x = row_of(a, r, ignored);
        const int kc = cols(x.keep), rc = cols(x.room);
        const unsigned plan = (unsigned)__ldcg(&a.at[r]);
        const int replace = (int)(plan >> 31);
        const int* fresh = a.free_ids + (plan & 0x7fffffffu) + replace - kc;  // the new page of column c is fresh[c]
        const int* held = a.page_table + (long long)x.parent * a.max_pages;   // read where c < kc only
        const bool first = x.parent >= 0 && __ldcg(&a.first[x.parent]) == r;
        for (int c = tid; c < a.max_pages; c += kApplyThreads) {
            int page = -1;
            if (c < kc - replace) {
                page = __ldcg(&held[c]);
                if (page < 0 || page >= a.P) bad |= kErrBadPage;
                else if (!first) atomicAdd(&a.refs_out[page], 1);
            } else if (c < rc) {
                page = __ldcg(&fresh[c]);
                a.refs_out[page] = 1;
            }
            out[c] = page;
        }
        if (tid == 0) {
            a.out_lens[r] = x.room;
            int src = -1, dst = -1, tokens = 0;
            if (replace) {
                src = __ldcg(&held[kc - 1]);
                dst = __ldcg(&fresh[kc - 1]);
                tokens = x.keep % kPageSize;
                if (first) atomicSub(&a.refs_out[src], 1);
            }
            a.copies[3ll * r] = src;
            a.copies[3ll * r + 1] = dst;
            a.copies[3ll * r + 2] = tokens;
        }
    } else if (ok) {
        const int p = (int)blockIdx.x - a.Rout;
        const int f = __ldcg(&a.first[p]);
        const int from = f == INT_MAX ? 0 : cols(row_of(a, f, ignored).keep), to = cols(held_of(a, p));
        const int* held = a.page_table + (long long)p * a.max_pages;
        for (int c = from + tid; c < to; c += kApplyThreads) {
            const int page = __ldcg(&held[c]);
            if (page < 0 || page >= a.P) bad |= kErrBadPage;
            else atomicSub(&a.refs_out[page], 1);
        }
    }
    if (bad) atomicOr(a.err, bad);
}

}  // namespace

size_t fork_workspace(int Rin, int Rout, int P) { return (size_t(Rin) * 3 + size_t(Rout) + size_t(P) + 1) * 4; }

cudaError_t pages_fork_launch(const ForkArgs& a, cudaStream_t stream) {
    // one CTA while a row or page or two per thread are all there is, else a cluster of eight
    const int most = a.Rin > a.Rout ? (a.Rin > a.P ? a.Rin : a.P) : (a.Rout > a.P ? a.Rout : a.P);
    const int ctas = most <= 2 * kPlanThreads ? 1 : 8;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaError_t e = cudaLaunchKernelEx(&cfg, fork_plan_kernel, a);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)(a.Rout + a.Rin));
    cfg.blockDim = dim3(kApplyThreads);
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fork_apply_kernel, a);
}

}  // namespace sinkattn
