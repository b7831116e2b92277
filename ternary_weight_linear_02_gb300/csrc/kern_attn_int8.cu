// kern_attn_int8.cu -- the attention kernels for caches in int8.
#include "attn_stream.cuh"

namespace tl {

cudaError_t launch_stream_int8(const AttnArgs &a, bool bf, int nc, cudaStream_t st) {
    return launch_stream<kKvInt8>(a, bf, nc, st);
}

}  // namespace tl
