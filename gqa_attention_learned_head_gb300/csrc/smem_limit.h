// smem_limit.h -- host side: the dynamic shared memory that a kernel may be launched with.  Internal to libsinkattn.
#pragma once
#include <cuda_runtime.h>

namespace sinkattn {

// Raises `kernel`'s limit to the most that a block may have on the current device, `dev`.  The limit belongs to the process:
// set to what one call needs, it would be lowered under another host thread's larger call.  done: the kernel's own flags, one per
// device, of the calling thread.
inline cudaError_t allow_all_smem(const void* kernel, int dev, bool (&done)[64]) {
    if (dev < 64 && done[dev]) return cudaSuccess;
    int most = 0;
    cudaFuncAttributes fa;
    cudaError_t e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, kernel);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most - (int)fa.sharedSizeBytes);
    if (e == cudaSuccess && dev < 64) done[dev] = true;
    return e;
}

}  // namespace sinkattn
