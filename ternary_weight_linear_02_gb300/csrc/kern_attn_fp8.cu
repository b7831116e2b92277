// kern_attn_fp8.cu -- the attention kernels for caches in fp8.
#include "attn_stream.cuh"

namespace tl {

cudaError_t launch_stream_fp8(const AttnArgs &a, bool bf, int nc, cudaStream_t st) {
    return launch_stream<kKvFp8>(a, bf, nc, st);
}

}  // namespace tl
