// cq_window.cu -- attention of drafted tokens over a sliding window and the first tokens of a paged cache.
#define CQ_TREE_WINDOW 1
#include "cq_tree_kernel.h"

namespace cq {

int launch_kv_window_attend(const cq_kv_geom &g, const cq_kv_tree &t, const cq_kv_window &w, const float *lk, const float *lv, void *stream) {
    TreeParams p;
    p.positions = w.positions, p.window = w.window, p.sinks = w.sinks, p.span = INT_MAX;
    const Shape s = shape_of(g, t.n_seqs, t.max_nodes, p.unit);
    if (in_line(s.N, w.positions, t.mask)) {
        p.span = 1;
        for (int i = 0; i < s.n_units; ++i) {
            const int rows = p.unit[i].nh * (g.n_q_heads / g.n_kv_heads);  // columns of a token
            p.span = std::max(p.span, s.N % rows ? (s.N + rows - 2) / rows + 1 : s.N / rows);
        }
    }
    return launch_attend(p, g, t, lk, lv, false, stream);
}

}  // namespace cq
