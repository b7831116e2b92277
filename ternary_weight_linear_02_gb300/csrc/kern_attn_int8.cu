// kern_attn_int8.cu -- the attention kernels for caches in int8.
#include "attn_stream.cuh"
#include "attn_tile.cuh"

namespace tl {

cudaError_t launch_attn_int8(const AttnArgs &a, bool tile, int sms, cudaStream_t st) {
    return tile ? launch_tile<kKvInt8>(a, sms, st) : launch_stream<kKvInt8>(a, sms, st);
}

}  // namespace tl
