// kern_attn_fp8.cu -- the attention kernels for caches in fp8.
#include "attn_stream.cuh"
#include "attn_tile.cuh"

namespace tl {

cudaError_t launch_attn_fp8(const AttnArgs &a, bool tile, int sms, cudaStream_t st) {
    return tile ? launch_tile<kKvFp8>(a, sms, st) : launch_stream<kKvFp8>(a, sms, st);
}

}  // namespace tl
