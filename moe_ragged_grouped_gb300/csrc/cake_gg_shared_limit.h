// cake_gg_shared_limit.h -- a kernel's opt-in limit of dynamic shared memory.
#pragma once

#include <atomic>
#include <cstddef>

#include <cuda_runtime.h>

namespace cakegg {

// Raises the limit of a kernel to `bytes` on the current device, the first time that it
// is asked there.  The limit is the kernel's, not the launch's: a caller asks for the most
// that any launch of the kernel takes, so that no thread's launch finds less than it needs
// because another thread set it for a smaller one.
template <auto KERNEL>
cudaError_t raise_shared_limit(size_t bytes)
{
    static std::atomic<bool> raised[64] = {};
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (raised[dev].load(std::memory_order_relaxed)) return cudaSuccess;
    err = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
    if (err == cudaSuccess) raised[dev].store(true, std::memory_order_relaxed);   // (set twice by two threads at once it is the same)
    return err;
}

}  // namespace cakegg
