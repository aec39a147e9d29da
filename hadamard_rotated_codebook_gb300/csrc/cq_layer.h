// cq_layer.h -- declarations shared by the translation units of a layer's other serving steps: block norms and
// low-rank adapters (cq_layer_host.cpp checks arguments and calls the launchers; each launcher lives in the .cu
// file of its kernel).
#pragma once

#include "cq_internal.h"

namespace cq {

int launch_block_norm(const cq_norm_desc &d, void *stream);

// A call of cq_lora_add as its kernels take it.
struct LoraParams {
    cq_lora_desc d;
    unsigned int *status;
    int cluster;  // blocks that share a piece of work
    bool vec_b;   // rows of B in runs of 4
    bool vec_y[CQ_LORA_MAX_MATS];  // rows of y likewise
};
// vec: rows of x and A in runs of 8.
int launch_lora_f16(LoraParams &p, bool vec, void *stream);
int launch_lora_bf16(LoraParams &p, bool vec, void *stream);

}  // namespace cq
