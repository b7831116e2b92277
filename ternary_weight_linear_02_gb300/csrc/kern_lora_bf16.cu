// kern_lora_bf16.cu -- the adapter kernel (kern_lora.cuh) for bf16 inputs.
#include "kern_lora.cuh"

namespace tl {
cudaError_t launch_lora_bf16(const LoraArgs &a, bool f32, bool big, int units, cudaStream_t st) {
    return lora::launch_type<__nv_bfloat16>(a, f32, big, units, st);
}
}  // namespace tl
