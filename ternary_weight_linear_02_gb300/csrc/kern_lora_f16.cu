// kern_lora_f16.cu -- the adapter kernel (kern_lora.cuh) for fp16 inputs.
#include "kern_lora.cuh"

namespace tl {
cudaError_t launch_lora_f16(const LoraArgs &a, bool f32, bool big, int units, cudaStream_t st) {
    return lora::launch_type<__half>(a, f32, big, units, st);
}
}  // namespace tl
