// cq_paged.h -- declarations shared by the translation units of the paged KV
// cache (cq_paged_host.cpp checks arguments and calls the launchers; each
// launcher lives in the .cu file of its kernel).
#pragma once

#include "cq_internal.h"

namespace cq {

int launch_qk_norm_rope(const cq_qk_desc &d, void *stream);
int launch_kv_plan(const cq_kv_step &s, void *stream);

// One cache of a slot write.
struct SlotSide {
    uint8_t *codes, *norms;  // the blob's two regions
    const void *rows;
    int64_t stride;          // elements between rows
    int width, groups, bits;
    const float *codebook;   // host
};
int launch_kv_write_slots(const SlotSide side[2], int cap, int dtype, const int32_t *slots, int n, void *stream);

// Key/value heads that are attended together: all of them share the key
// groups gk .. gk + ngk - 1 and the value groups gv .. gv + ngv - 1 of a cache
// row, so one pass over those groups' codes serves every query head of the unit.
constexpr int kMaxUnits = 128;
struct TreeUnit {
    short h0, nh;  // key/value heads h0 .. h0 + nh - 1
    short gk, ngk, gv, ngv;
};
// Units of a geometry: consecutive heads are joined while they add no group.
// Returns their number, or 0 if a head spans more than two groups or there
// are too many.
int tree_units(const cq_kv_geom &g, TreeUnit *u);

// Whether the attention's shared-memory layout holds on a device that keeps `reserved` bytes of each block's shared memory for
// itself: CQ_OK, or the error that the call returns before it launches anything.
int tree_smem_check(int reserved);
size_t tree_workspace(const cq_kv_geom &g, int n_seqs, int max_nodes);
// lk, lv: level tables of the key and value codes (level_table).
// give_up: nobody tells the products that the queries are there, and waits give up after a few polls (a self-test).
int launch_kv_tree_attend(const cq_kv_geom &g, const cq_kv_tree &t, const float *lk, const float *lv, bool give_up, void *stream);

}  // namespace cq
