// kv_unpack_q8.cu -- pages of a cache held in 8 bits as bf16 pages: code x scale, which bf16 holds exactly (4 significant bits).
//
// Both kernels are bound by HBM: a byte in and two out a value, the two scales of a (page, KV head) in 2 bytes.  A warp takes one
// (page, KV head): its keys and values are contiguous 1 KiB slices, read 8 codes a lane, all loads issued before the first store, so
// that every store instruction writes 512 contiguous bytes.  Measured (GB300): 8192 pages of 8 KV heads (403 MB) 59.5 us, 6.8 TB/s, the
// copy rate; 130 pages 2.4 us, latency.
//   unpack_q8_kernel  a list of (source page, destination page, tokens), as sinkattn_kv_copy takes it;
//   widen_q8_kernel   every page that the sequences of a prefill hold, found on the device from their lengths: the work is the
//                     flattened list of (sequence, page, KV head), cut into equal shares, one a warp.
#include "args_q8.h"
#include "ptx.cuh"
#include "q8.cuh"
#include "smem_limit.h"

namespace sinkattn {
namespace {

constexpr int kWarps = 8;

// The first `tokens` tokens of a slice of keys and of values, as bf16.
__device__ __forceinline__ void widen_slice(const uint8_t* k, const uint8_t* v, const uint8_t* scales, __nv_bfloat16* k_out,
                                            __nv_bfloat16* v_out, int tokens, int lane, unsigned* err) {
    const int pieces = tokens * (kHeadDim / 8);
    const uint2 *ks = reinterpret_cast<const uint2*>(k), *vs = reinterpret_cast<const uint2*>(v);
    uint2 x[4], y[4];
    const uint32_t sc = __ldcg(reinterpret_cast<const unsigned short*>(scales));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (lane + 32 * j < pieces) {
            x[j] = __ldcg(ks + lane + 32 * j);
            y[j] = __ldcg(vs + lane + 32 * j);
        }
    }
    bool off = false;
    const float fk = q8::power(q8::scale_byte(sc & 0xFF, off)), fv = q8::power(q8::scale_byte(sc >> 8, off));
    if (off && lane == 0) atomicOr(err, kErrBadValue);
    uint4 *ko = reinterpret_cast<uint4*>(k_out), *vo = reinterpret_cast<uint4*>(v_out);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (lane + 32 * j < pieces) {
            ko[lane + 32 * j] = q8::widen8(x[j], fk);
            vo[lane + 32 * j] = q8::widen8(y[j], fv);
        }
    }
}

constexpr int kSlice = kPageSize * kHeadDim;  // values of one (page, KV head)

__global__ void __launch_bounds__(kWarps * 32) unpack_q8_kernel(const UnpackQ8Args a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const long long unit = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);  // (entry, head), head fastest
    const int g = (int)(unit % a.Hkv);
    const long long i = unit / a.Hkv;
    if (i >= a.n) return;
    const int src = __ldcg(&a.copies[3 * i]), dst = __ldcg(&a.copies[3 * i + 1]);
    int tokens = __ldcg(&a.copies[3 * i + 2]);
    if (src == -1 && dst == -1) return;
    const bool report = lane == 0 && g == 0;
    if (src < 0 || src >= a.P || dst < 0 || dst >= a.P_out) {
        if (report) atomicOr(a.err, kErrBadPage);
        return;
    }
    if (tokens < 0 || tokens > kPageSize) {
        if (report) atomicOr(a.err, kErrBadLength);
        tokens = tokens < 0 ? 0 : kPageSize;
    }
    if (tokens == 0) return;
    const long long from = (long long)src * a.Hkv + g, to = (long long)dst * a.Hkv + g;
    widen_slice(a.k_pages + from * kSlice, a.v_pages + from * kSlice, a.kv_scales + from * 2, a.k_out + to * kSlice,
                a.v_out + to * kSlice, tokens, lane, a.err);
}

// Cached tokens of sequence n once its new ones are in, as the prefill over the pages counts them.
__device__ __forceinline__ int kv_total(const WidenQ8Args& a, int n) {
    const long long cap = (long long)a.max_pages * kPageSize;
    const int c0 = __ldg(&a.cu_seqlens[n]), c1 = __ldg(&a.cu_seqlens[n + 1]);
    if (c0 < 0 || c1 <= c0 || c1 > a.T) return 0;
    const long long L = min(c1 - c0, a.max_seqlen);
    long long s = __ldg(&a.start_pos[n]);
    s = s < 0 ? 0 : s;
    return (int)min(s + L, cap);
}

__global__ void __launch_bounds__(kWarps * 32) widen_q8_kernel(const WidenQ8Args a) {
    extern __shared__ int prefix[];  // [N + 1] pages before each sequence
    __shared__ int sums[kWarps];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int running = 0;
    for (int base = 0; base < a.N; base += kWarps * 32) {
        const int n = base + tid;
        const int pages = n < a.N ? (kv_total(a, n) + kPageSize - 1) / kPageSize : 0;
        int incl = pages;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) sums[warp] = incl;
        __syncthreads();
        int before = 0, total = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            before += w < warp ? sums[w] : 0;
            total += sums[w];
        }
        if (n < a.N) prefix[n] = running + before + incl - pages;
        running += total;
        __syncthreads();
    }
    if (tid == 0) prefix[a.N] = running;
    __syncthreads();
    const long long U = (long long)running * a.Hkv, W = (long long)gridDim.x * kWarps;
    const long long w = (long long)blockIdx.x * kWarps + warp;
    const long long u0 = w * U / W, u1 = (w + 1) * U / W;
    if (u0 < u1) {
        int lo = 0, hi = a.N - 1;  // the sequence of the share's first page: smallest n with prefix[n + 1] > page
        const int first = (int)(u0 / a.Hkv);
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (prefix[mid + 1] > first) hi = mid;
            else lo = mid + 1;
        }
        int n = lo;
        for (long long u = u0; u < u1; ++u) {
            const int p = (int)(u / a.Hkv), g = (int)(u - (long long)p * a.Hkv);
            while (prefix[n + 1] <= p) ++n;
            const long long at = (long long)n * a.max_pages + (p - prefix[n]);
            const int src = __ldg(&a.page_table[at]);
            const bool ok = src >= 0 && src < a.num_pages;  // (the prefill reports a page id that is not)
            if (a.remap && g == 0 && lane == 0) a.remap[at] = ok ? (int)at : -1;
            if (!ok) continue;
            const long long from = (long long)src * a.Hkv + g, to = a.remap ? at * a.Hkv + g : from;
            widen_slice(a.k_pages + from * kSlice, a.v_pages + from * kSlice, a.kv_scales + from * 2, a.k_out + to * kSlice,
                        a.v_out + to * kSlice, kPageSize, lane, a.err);
        }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

void dependent(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, unsigned grid, cudaStream_t stream) {
    attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr->val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
}

}  // namespace

cudaError_t unpack_q8_launch(const UnpackQ8Args& a, cudaStream_t stream) {
    const long long blocks = ((long long)a.n * a.Hkv + kWarps - 1) / kWarps;
    if (blocks == 0) return cudaSuccess;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = {};
    dependent(cfg, attr, (unsigned)blocks, stream);
    return cudaLaunchKernelEx(&cfg, unpack_q8_kernel, a);
}

cudaError_t widen_q8_launch(const WidenQ8Args& a, cudaStream_t stream) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    static thread_local bool done[64] = {};
    const size_t smem = (size_t)(a.N + 1) * sizeof(int);
    if (smem > 40000 && (e = allow_all_smem(reinterpret_cast<const void*>(widen_q8_kernel), dev, done)) != cudaSuccess) return e;
    // eight CTAs an SM (six run at once, at 40 registers), fewer where the tables cannot hold a page for each warp
    const long long most = ((long long)a.N * a.max_pages * a.Hkv + kWarps - 1) / kWarps;
    const long long resident = (long long)sms * (smem > 24000 ? 3 : 8);
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = {};
    dependent(cfg, attr, (unsigned)(most < resident ? most : resident), stream);
    cfg.dynamicSmemBytes = smem;
    return cudaLaunchKernelEx(&cfg, widen_q8_kernel, a);
}

}  // namespace sinkattn
