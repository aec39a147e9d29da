// cq_window.cu -- attention of drafted tokens over a sliding window and the first tokens of a paged cache.
#define CQ_TREE_WINDOW 1
#include "cq_tree_kernel.h"

namespace cq {

int launch_kv_window_attend(const cq_kv_geom &g, const cq_kv_tree &t, const cq_kv_window &w, const float *lk, const float *lv, void *stream) {
    TreeParams p;
    p.positions = w.positions, p.window = w.window, p.sinks = w.sinks;
    return launch_attend(p, g, t, lk, lv, false, stream);
}

}  // namespace cq
