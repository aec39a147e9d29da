// cq_layer.h -- declarations shared by the translation units of a layer's other serving steps: block norms and
// low-rank adapters (cq_layer_host.cpp checks arguments and calls the launchers; each launcher lives in the .cu
// file of its kernel).
#pragma once

#include "cq_internal.h"

namespace cq {

// give_up: the kernel waits for what never lands, and a few polls at most (a self-test).
int launch_block_norm(const cq_norm_desc &d, bool give_up, void *stream);

// A call of cq_lora_add as its kernels take it.
constexpr int kMaxSplits = 8;
struct LoraParams {
    cq_lora_desc d;
    unsigned int *status;
    float *u;      // the workspace: what the blocks of the first product leave, [matrix][part][token][u_row]
    int u_row;     // ranks, rounded up to what a block sums
    int pieces;    // of up to so many tokens of a request as a block takes, at most
    int splits;    // parts of k
    int runs;      // of 32 outputs that a warp of the second product takes
    bool few;      // pieces of 8: few tokens a request, or few in all
    bool vec;      // rows of x and A in runs of 8
    bool tensor;   // x and A by tensor copies: rows on 16 bytes, and no fp32
    bool vec_b;    // rows of B in runs of 4
    bool vec_y[CQ_LORA_MAX_MATS];  // rows of y likewise
    unsigned spin;  // polls after which a wait gives up
    bool give_up;   // the kernels on tcgen05 wait for what never ends, and a few polls at most (a self-test)
};
// Tiles of 16 ranks that a block of the first product takes.
constexpr int lora_rank_tiles(int rank) { return rank <= 16 ? 1 : rank <= 32 ? 2 : 4; }
// Tokens of a piece, by the activations' type and the tiles of ranks: 8 where requests have few, else as many as leave the
// sums in registers and two stages of inputs in shared memory; 128 by tensor copies. And the warps that share them.
constexpr int lora_tokens(int x_dtype, int tiles, bool few, bool tensor) {
    return few ? 8 : tensor ? 128 : tiles == 4 ? (x_dtype == CQ_T_F32 ? 32 : 64) : tiles == 2 || x_dtype == CQ_T_F32 ? 64 : 128;
}
constexpr int lora_warps_along(bool few) { return few ? 1 : 2; }
int launch_lora_f16(LoraParams &p, void *stream);
int launch_lora_bf16(LoraParams &p, void *stream);

}  // namespace cq
