// launch.h -- what launchers share.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace tl {

// Raises a kernel's limit of dynamic shared memory on the current device, once per device: a bit of `done`
// each, set only after the call succeeded.
template <typename K>
cudaError_t allow_smem(std::atomic<uint64_t> &done, K *kernel, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

}  // namespace tl
