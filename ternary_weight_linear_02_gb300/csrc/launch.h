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

// A launch that may begin while the kernel before it in the stream ends: the kernel calls pdl_wait() before it touches
// anything.  cluster: blocks of a cluster (0: none).
template <typename... P, typename... A>
cudaError_t launch_chained(void (*kernel)(P...), unsigned blocks, unsigned threads, size_t smem, unsigned cluster, cudaStream_t st,
                           const A &...args) {
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(blocks);
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    c.attrs = at;
    c.numAttrs = cluster ? 2 : 1;
    return cudaLaunchKernelEx(&c, kernel, P(args)...);
}

}  // namespace tl
