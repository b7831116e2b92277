// api_util.h -- what the C ABI files for rotation, cache, attention and serving share.
#pragma once

#include "kernels.h"
#include "ternary_linear.h"

namespace tl {

inline bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

inline tl_status from_cuda(cudaError_t e) {
    if (e == cudaSuccess) return TL_OK;
    cudaGetLastError();
    return TL_ERR_CUDA;
}

// Offsets stay far inside 63 bits: |stride| < 2^40, axis < 2^31 in any use.
inline bool stride_ok(int64_t s) { return s > -((int64_t)1 << 40) && s < ((int64_t)1 << 40); }

tl_status check_cache(const tl_kv_cache *c, KvCache *out);  // api_attn.cu

}  // namespace tl
