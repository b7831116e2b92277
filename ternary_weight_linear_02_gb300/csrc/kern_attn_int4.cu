// kern_attn_int4.cu -- the attention kernels for caches in int4.
#include "attn_stream.cuh"
#include "attn_tile.cuh"

namespace tl {

cudaError_t launch_attn_int4(const AttnArgs &a, bool tile, int sms, cudaStream_t st) {
    return tile ? launch_tile<kKvInt4>(a, sms, st) : launch_stream<kKvInt4>(a, sms, st);
}

}  // namespace tl
