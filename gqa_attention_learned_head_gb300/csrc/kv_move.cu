// kv_move.cu -- copies of pages, and the compaction of accepted draft tokens, inside the K/V pools of one
// or several layers.
//
// Both move 128-byte rows (one token of one KV head) and compute nothing: bound by HBM, one read and one
// write of what moves.  A warp takes one (entry, layer, KV head): its rows of K and of V are contiguous
// 2 KB slices of the pools, read with 16-byte loads that are all issued before the first store, so a warp
// has up to 4 KB in flight (and a compaction may overwrite its own sources).
//
// Measured (GB300): 4096 whole pages of 8 KV heads (268 MB moved) 41.8 us, 6.4 TB/s = 95% of the copy rate; 16
// accepted tokens of 256 requests in 24 layers (214 MB) 32.5 us, 6.6 TB/s = 97%; 256 tails of a page 2.8 us, 32 trees
// of 8 tokens 2.2 us, both little more than the latency of one kernel.
#include "args_pages.h"
#include "errors_beam.h"
#include "ptx.cuh"

namespace sinkattn {
namespace {

constexpr int kWarps = 8;

__global__ void __launch_bounds__(kWarps * 32) kv_copy_kernel(const CopyArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const long long unit = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);  // (layer, entry, head), head fastest
    const int g = (int)(unit % a.Hkv);
    const long long le = unit / a.Hkv;
    const int i = (int)(le % a.n), layer = (int)(le / a.n);
    if (layer >= a.L) return;
    const int src = __ldcg(&a.copies[3ll * i]), dst = __ldcg(&a.copies[3ll * i + 1]);
    int tokens = __ldcg(&a.copies[3ll * i + 2]);
    if (src == -1 && dst == -1) return;
    const bool report = lane == 0 && g == 0 && layer == 0;
    if (src < 0 || src >= a.P || dst < 0 || dst >= a.P) {
        if (report) atomicOr(a.err, kErrBadPage);
        return;
    }
    if (tokens < 0 || tokens > kPageSize) {
        if (report) atomicOr(a.err, kErrBadLength);
        tokens = tokens < 0 ? 0 : kPageSize;
    }
    const long long base = (long long)layer * a.P;
    const long long from = ((base + src) * a.Hkv + g) * (kPageSize * kHeadDim / 8);  // in 16-byte pieces
    const long long to = ((base + dst) * a.Hkv + g) * (kPageSize * kHeadDim / 8);
    uint4* k = reinterpret_cast<uint4*>(a.k_pages);
    uint4* v = reinterpret_cast<uint4*>(a.v_pages);
    const int pieces = tokens * (kHeadDim / 8);
    uint4 x[4], y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int p = lane + 32 * j;
        if (p < pieces) {
            x[j] = k[from + p];
            y[j] = v[from + p];
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int p = lane + 32 * j;
        if (p < pieces) {
            k[to + p] = x[j];
            v[to + p] = y[j];
        }
    }
}

__global__ void __launch_bounds__(kWarps * 32) kv_compact_kernel(const CompactArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const long long unit = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);  // (layer, request, head), head fastest
    const int g = (int)(unit % a.Hkv);
    const long long lb = unit / a.Hkv;
    const int b = (int)(lb % a.B), layer = (int)(lb / a.B);
    if (layer >= a.L) return;
    const bool report = g == 0 && layer == 0;
    int n = __ldcg(&a.num_accepted[b]);
    if (n < 0 || n > a.A) {
        if (report && lane == 0) atomicOr(a.err, kErrBadLength);
        n = n < 0 ? 0 : a.A;
    }
    const long long start = __ldcg(&a.start_pos[b]), cap = (long long)a.max_pages * kPageSize;
    const int* table = a.page_table + (long long)b * a.max_pages;
    // lane i < n finds where token i comes from and goes to, as rows of the layer's pool
    long long from = -1, to = -1;
    if (lane < n) {
        const int idx = __ldcg(&a.accepted[(long long)b * a.A + lane]);
        const long long ps = start + idx, pd = start + lane;
        if (idx < 0) {
            if (report) atomicOr(a.err, kErrBadIndex);
        } else if (pd < 0 || ps < 0 || ps >= cap || pd >= cap) {
            if (report) atomicOr(a.err, kErrBadLength);
        } else if (idx != lane) {
            const int s = __ldcg(&table[ps / kPageSize]), d = __ldcg(&table[pd / kPageSize]);
            if (s < 0 || s >= a.P || d < 0 || d >= a.P) {
                if (report) atomicOr(a.err, kErrBadPage);
            } else {
                const long long base = (long long)layer * a.P;
                from = ((base + s) * a.Hkv + g) * kPageSize + ps % kPageSize;
                to = ((base + d) * a.Hkv + g) * kPageSize + pd % kPageSize;
            }
        }
    }
    // eight lanes a row, four rows at a time
    uint4* k = reinterpret_cast<uint4*>(a.k_pages);
    uint4* v = reinterpret_cast<uint4*>(a.v_pages);
    uint4 x[kMaxAccepted / 4], y[kMaxAccepted / 4];
    long long dst[kMaxAccepted / 4];
#pragma unroll
    for (int j = 0; j < kMaxAccepted / 4; ++j) {
        const long long src = __shfl_sync(0xffffffffu, from, 4 * j + lane / 8);
        dst[j] = __shfl_sync(0xffffffffu, to, 4 * j + lane / 8);
        if (dst[j] >= 0) {
            x[j] = k[src * 8 + lane % 8];
            y[j] = v[src * 8 + lane % 8];
        }
    }
    __syncwarp();  // every lane has its pieces before any row is overwritten
#pragma unroll
    for (int j = 0; j < kMaxAccepted / 4; ++j) {
        if (dst[j] >= 0) {
            k[dst[j] * 8 + lane % 8] = x[j];
            v[dst[j] * 8 + lane % 8] = y[j];
        }
    }
}

template <class Args>
cudaError_t launch_units(void (*kernel)(const Args), const Args& a, long long units, cudaStream_t stream) {
    const long long blocks = (units + kWarps - 1) / kWarps;
    if (blocks == 0) return cudaSuccess;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t kv_copy_launch(const CopyArgs& a, cudaStream_t stream) {
    return launch_units(kv_copy_kernel, a, (long long)a.L * a.n * a.Hkv, stream);
}

cudaError_t kv_compact_launch(const CompactArgs& a, cudaStream_t stream) {
    return launch_units(kv_compact_kernel, a, (long long)a.L * a.B * a.Hkv, stream);
}

}  // namespace sinkattn
