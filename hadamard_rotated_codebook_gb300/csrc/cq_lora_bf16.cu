// cq_lora_bf16.cu -- the adapter kernels of bf16 weights.
#include "cq_lora_kernel.h"

namespace cq {

int launch_lora_bf16(LoraParams &p, void *stream) { return launch_t<__nv_bfloat16>(p, reinterpret_cast<cudaStream_t>(stream)); }

}  // namespace cq
