// kern_attn_int4.cu -- the attention kernels for caches in int4.
#include "attn_stream.cuh"

namespace tl {

cudaError_t launch_stream_int4(const AttnArgs &a, bool bf, int nc, cudaStream_t st) {
    return launch_stream<kKvInt4>(a, bf, nc, st);
}

}  // namespace tl
