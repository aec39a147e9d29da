// cq_lora_f16.cu -- the adapter kernels of fp16 weights (a translation unit per weight type, so that they compile side by side).
#include "cq_lora_kernel.h"

namespace cq {

int launch_lora_f16(LoraParams &p, void *stream) { return launch_t<__half>(p, reinterpret_cast<cudaStream_t>(stream)); }

}  // namespace cq
