// cq_tree.cu -- attention of drafted tokens over a whole paged cache: the kernel, and what its launch shares with the windowed one.
#define CQ_TREE_WINDOW 0
#include "cq_tree_kernel.h"

namespace cq {

int tree_smem_check(int reserved) {
    if (reserved == kSmemFirst) return CQ_OK;
    return set_error(CQ_ERR_CUDA, "tree attention counts on shared memory from byte %d on, and the system keeps %d bytes", kSmemFirst, reserved);
}

size_t tree_workspace(const cq_kv_geom &g, int n_seqs, int max_nodes) {
    if (!n_seqs || !max_nodes) return 0;
    TreeUnit u[kMaxUnits];
    const Shape s = shape_of(g, n_seqs, max_nodes, u);
    return up16(s.items * sizeof(int2)) + up16(s.slots * s.N * sizeof(float2)) + s.slots * s.ng * s.N * kGroup * sizeof(float);
}

int launch_kv_tree_attend(const cq_kv_geom &g, const cq_kv_tree &t, const float *lk, const float *lv, bool give_up, void *stream) {
    TreeParams p;
    return launch_attend(p, g, t, lk, lv, give_up, stream);
}

}  // namespace cq
