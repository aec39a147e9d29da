// cq_paged_host.cpp -- host side of the paged KV cache's entry points:
// argument checks, the rotation rates, the units of a geometry.
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "cq_paged.h"

using namespace cq;

namespace {

constexpr int kMaxRowWidth = 1 << 16;  // elements of a cache row

bool overlap(const void *a, uint64_t na, const void *b, uint64_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

// x without its whole part as a 64-bit binary fraction, modulo 1.
uint64_t fraction(double x) {
    x -= std::trunc(x);
    const uint64_t v = (uint64_t)(std::fabs(x) * 18446744073709551616.0);  // below 2^64: x is exact and below 1
    return x < 0 ? 0 - v : v;
}
// f / (2 pi) modulo 1. The quotient in 64 bits alone is off by up to 2^-53 of itself, which a position of 10^9 makes more than
// fp32's part in the angle; its remainder (2 pi in two doubles) brings the rest.
uint64_t turns(double f) {
    const double hi = 6.283185307179586, lo = 2.4492935982947064e-16;
    const double q = f / hi;
    return fraction(q) + fraction(std::fma(-q, lo, std::fma(-q, hi, f)) / hi);
}

// What the slot write and the attention need of a geometry.
int check_cache_geom(const cq_kv_geom *g) {
    if (!g) return set_error(CQ_ERR_ARG, "null geometry");
    if (g->n_kv_heads < 1 || g->head_dim_k < 1 || g->head_dim_v < 1 ||
        (int64_t)g->n_kv_heads * g->head_dim_k > kMaxRowWidth || (int64_t)g->n_kv_heads * g->head_dim_v > kMaxRowWidth)
        return set_error(CQ_ERR_SHAPE, "cache rows of %d x %d (keys) and %d x %d (values) exceed %d or are empty",
                         g->n_kv_heads, g->head_dim_k, g->n_kv_heads, g->head_dim_v, kMaxRowWidth);
    if (width_of(g->k_bits) < 2 || width_of(g->v_bits) < 2)
        return set_error(CQ_ERR_ARG, "bits must be 2, 3, 4 or 5 (got %d, %d)", g->k_bits, g->v_bits);
    int st = check_codebook(g->k_codebook, g->k_bits);
    return st ? st : check_codebook(g->v_codebook, g->v_bits);
}

int check_tree_geom(const cq_kv_geom *g, TreeUnit *u) {
    int st = check_cache_geom(g);
    if (st) return st;
    if (g->n_q_heads < 1 || g->n_q_heads % g->n_kv_heads || g->n_q_heads > 1024)
        return set_error(CQ_ERR_SHAPE, "need 1..1024 query heads, a multiple of the %d key/value heads; got %d",
                         g->n_kv_heads, g->n_q_heads);
    if (!std::isfinite(g->scale)) return set_error(CQ_ERR_ARG, "scale must be finite");
    if (!tree_units(*g, u))
        return set_error(CQ_ERR_SHAPE,
                         "head widths %d (keys) and %d (values) over %d heads: a head spans more than two groups of 128, "
                         "or there are over %d groups", g->head_dim_k, g->head_dim_v, g->n_kv_heads, kMaxUnits);
    return CQ_OK;
}

}  // namespace

namespace cq {

int tree_units(const cq_kv_geom &g, TreeUnit *u) {
    int n = 0;
    for (int h = 0; h < g.n_kv_heads;) {
        const int gk = h * g.head_dim_k / kGroup, gv = h * g.head_dim_v / kGroup;
        auto span_k = [&](int end) { return (end * g.head_dim_k + kGroup - 1) / kGroup - gk; };
        auto span_v = [&](int end) { return (end * g.head_dim_v + kGroup - 1) / kGroup - gv; };
        const int ngk = span_k(h + 1), ngv = span_v(h + 1);
        if (ngk > 2 || ngv > 2 || n == kMaxUnits) return 0;
        int e = h + 1;
        while (e < g.n_kv_heads && span_k(e + 1) <= ngk && span_v(e + 1) <= ngv) ++e;
        u[n].h0 = (short)h;
        u[n].nh = (short)(e - h);
        u[n].gk = (short)gk;
        u[n].ngk = (short)ngk;
        u[n].gv = (short)gv;
        u[n].ngv = (short)ngv;
        ++n;
        h = e;
    }
    return n;
}

}  // namespace cq

extern "C" {

int cq_rope_init(int rot_dim, double theta, const double *inv_freq, uint64_t *rates, size_t cap, size_t *n_rates) {
    clear_error();
    if (rot_dim < 0 || (rot_dim & 1) || rot_dim > 256)
        return set_error(CQ_ERR_SHAPE, "rot_dim must be even and 0..256, got %d", rot_dim);
    const int n = rot_dim / 2;
    if (n_rates) *n_rates = (size_t)n;
    if (!rates) return CQ_OK;
    if (cap < (size_t)n) return set_error(CQ_ERR_ARG, "need room for %d rates, got %zu", n, cap);
    if (!inv_freq && !(std::isfinite(theta) && theta > 0))
        return set_error(CQ_ERR_ARG, "theta must be positive and finite");
    for (int i = 0; i < n; ++i) {
        const double f = inv_freq ? inv_freq[i] : std::pow(theta, -2.0 * i / rot_dim);
        if (!std::isfinite(f)) return set_error(CQ_ERR_ARG, "inv_freq[%d] is not finite", i);
        rates[i] = turns(f);
    }
    return CQ_OK;
}

int cq_qk_norm_rope(const cq_qk_desc *d, void *stream) {
    clear_error();
    if (!d) return set_error(CQ_ERR_ARG, "null descriptor");
    for (int t : {d->in_dtype, d->q_out_dtype, d->k_out_dtype})
        if (t < CQ_T_F32 || t > CQ_T_BF16) return set_error(CQ_ERR_ARG, "unknown element type %d", t);
    if (d->head_dim < 2 || d->head_dim > 256 || (d->head_dim & 1))
        return set_error(CQ_ERR_SHAPE, "head_dim must be even and 2..256, got %d", d->head_dim);
    if (d->rot_dim < 0 || d->rot_dim > d->head_dim || (d->rot_dim & 1))
        return set_error(CQ_ERR_SHAPE, "rot_dim must be even and 0..head_dim (%d), got %d", d->head_dim, d->rot_dim);
    if (d->n_tokens < 0 || d->n_q_heads < 0 || d->n_kv_heads < 0 || (int64_t)d->n_q_heads + d->n_kv_heads > 65535)
        return set_error(CQ_ERR_SHAPE, "bad sizes: %d tokens, %d and %d heads", d->n_tokens, d->n_q_heads, d->n_kv_heads);
    if (!(d->eps >= 0) || !std::isfinite(d->eps) || !std::isfinite(d->weight_offset))
        return set_error(CQ_ERR_ARG, "eps must be finite and not negative, weight_offset finite");
    if (d->n_tokens == 0 || d->n_q_heads + d->n_kv_heads == 0) return CQ_OK;
    if ((d->n_q_heads && (!d->q || !d->q_out)) || (d->n_kv_heads && (!d->k || !d->k_out)))
        return set_error(CQ_ERR_ARG, "null q, k or output");
    if (d->rot_dim && (!d->rates || !d->positions)) return set_error(CQ_ERR_ARG, "null rates or positions");
    return launch_qk_norm_rope(*d, stream);
}

int cq_kv_plan(const cq_kv_step *s, void *stream) {
    clear_error();
    if (!s) return set_error(CQ_ERR_ARG, "null step");
    if (s->n_seqs < 0 || s->max_blocks < 0 || s->free_cap < 0 || s->n_tokens < 0)
        return set_error(CQ_ERR_SHAPE, "negative size");
    if (s->n_seqs > 1 << 20) return set_error(CQ_ERR_SHAPE, "at most %d requests, got %d", 1 << 20, s->n_seqs);
    if (s->block_size < 1) return set_error(CQ_ERR_SHAPE, "block_size must be at least 1, got %d", s->block_size);
    if (s->table_stride < s->max_blocks)
        return set_error(CQ_ERR_SHAPE, "table rows of %d blocks are %lld apart", s->max_blocks, (long long)s->table_stride);
    if (!s->cu_new || !s->n_free || !s->n_free_out) return set_error(CQ_ERR_ARG, "null cu_new, n_free or n_free_out");
    if (s->n_seqs && (!s->seq_lens || !s->new_lens || !s->held || !s->held_out))
        return set_error(CQ_ERR_ARG, "null seq_lens, new_lens, held or held_out");
    if (s->n_seqs && s->max_blocks && !s->block_table) return set_error(CQ_ERR_ARG, "null block_table");
    if (s->free_cap && !s->free_list) return set_error(CQ_ERR_ARG, "null free_list");
    if (s->n_tokens && (!s->slots || !s->positions || !s->token_seq))
        return set_error(CQ_ERR_ARG, "null slots, positions or token_seq");
    const uint64_t nb = (uint64_t)s->n_seqs * 4;
    if (s->n_free == s->n_free_out || (nb && overlap(s->held, nb, s->held_out, nb)))
        return set_error(CQ_ERR_ARG, "held_out and n_free_out must not be held and n_free themselves");
    return launch_kv_plan(*s, stream);
}

int cq_kv_write_slots(const cq_kv_geom *g, uint8_t *k_cache, uint8_t *v_cache, int cap, const void *k, int64_t k_stride,
                      const void *v, int64_t v_stride, int dtype, const int32_t *slots, int n, void *stream) {
    clear_error();
    int st = check_cache_geom(g);
    if (st) return st;
    if (dtype < CQ_T_F32 || dtype > CQ_T_BF16) return set_error(CQ_ERR_ARG, "unknown element type %d", dtype);
    if (cap < 0 || n < 0) return set_error(CQ_ERR_SHAPE, "negative size");
    if (n == 0) return CQ_OK;
    if (!slots || !k || !v) return set_error(CQ_ERR_ARG, "null rows or slots");
    if (cap > 0 && (!k_cache || !v_cache)) return set_error(CQ_ERR_ARG, "null cache");
    if ((reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache)) & 15)
        return set_error(CQ_ERR_ARG, "caches must be 16-byte aligned");
    SlotSide side[2];
    for (int i = 0; i < 2; ++i) {
        SlotSide &s = side[i];
        s.width = g->n_kv_heads * (i ? g->head_dim_v : g->head_dim_k);
        s.bits = i ? g->v_bits : g->k_bits;
        s.codebook = i ? g->v_codebook : g->k_codebook;
        s.groups = in_padded(s.width) / kGroup;
        s.rows = i ? v : k;
        s.stride = i ? v_stride : k_stride;
        s.codes = i ? v_cache : k_cache;
        s.norms = s.codes + (size_t)cap * s.groups * 16 * width_of(s.bits);
        if (s.stride < s.width && n > 1)
            return set_error(CQ_ERR_SHAPE, "rows of %d elements are %lld apart", s.width, (long long)s.stride);
    }
    return launch_kv_write_slots(side, cap, dtype, slots, n, stream);
}

int cq_selftest_tree_smem(int reserved) {
    clear_error();
    return tree_smem_check(reserved);
}

size_t cq_kv_tree_workspace(const cq_kv_geom *g, int n_seqs, int max_nodes) {
    clear_error();
    TreeUnit u[kMaxUnits];
    if (check_tree_geom(g, u)) return 0;
    if (n_seqs < 0 || max_nodes < 0 || max_nodes > CQ_TREE_MAX_NODES) {
        set_error(CQ_ERR_SHAPE, "bad sizes: %d requests of up to %d drafted tokens", n_seqs, max_nodes);
        return 0;
    }
    return tree_workspace(*g, n_seqs, max_nodes);
}

static int tree_attend(const cq_kv_geom *g, const cq_kv_tree *t, bool give_up, void *stream) {
    clear_error();
    TreeUnit u[kMaxUnits];
    int st = check_tree_geom(g, u);
    if (st) return st;
    if (!t) return set_error(CQ_ERR_ARG, "null tree");
    if (t->dtype != CQ_T_F16 && t->dtype != CQ_T_BF16)
        return set_error(CQ_ERR_ARG, "q and o are fp16 or bf16, got element type %d", t->dtype);
    if (t->n_seqs < 0 || t->n_nodes < 0 || t->cap < 0 || t->max_blocks < 0)
        return set_error(CQ_ERR_SHAPE, "negative size");
    if (t->max_nodes < 0 || t->max_nodes > CQ_TREE_MAX_NODES)
        return set_error(CQ_ERR_SHAPE, "at most %d drafted tokens per request, got %d", CQ_TREE_MAX_NODES, t->max_nodes);
    if (t->block_size < 1) return set_error(CQ_ERR_SHAPE, "block_size must be at least 1, got %d", t->block_size);
    if (t->table_stride < t->max_blocks)
        return set_error(CQ_ERR_SHAPE, "table rows of %d blocks are %lld apart", t->max_blocks, (long long)t->table_stride);
    if (t->mask && t->mask_words < (t->max_nodes + 31) / 32)
        return set_error(CQ_ERR_SHAPE, "%d mask words hold fewer than %d bits", t->mask_words, t->max_nodes);
    if (t->n_seqs == 0 || t->n_nodes == 0 || t->max_nodes == 0) return CQ_OK;
    if (!t->q || !t->o || !t->context_lens || !t->cu_nodes) return set_error(CQ_ERR_ARG, "null q, o, context_lens or cu_nodes");
    if (t->max_blocks && !t->block_table) return set_error(CQ_ERR_ARG, "null block_table");
    if (t->cap && (!t->k_cache || !t->v_cache)) return set_error(CQ_ERR_ARG, "null cache");
    if ((reinterpret_cast<uintptr_t>(t->k_cache) | reinterpret_cast<uintptr_t>(t->v_cache)) & 15)
        return set_error(CQ_ERR_ARG, "caches must be 16-byte aligned");
    const size_t need = tree_workspace(*g, t->n_seqs, t->max_nodes);
    if (need && (!t->workspace || t->workspace_bytes < need || (reinterpret_cast<uintptr_t>(t->workspace) & 15)))
        return set_error(CQ_ERR_ARG, "workspace of %zu bytes needed (16-byte aligned), got %zu", need,
                         t->workspace ? t->workspace_bytes : 0);
    float lk[16], lv[16];
    level_table(g->k_bits, g->k_codebook, lk);
    level_table(g->v_bits, g->v_codebook, lv);
    return launch_kv_tree_attend(*g, *t, lk, lv, give_up, stream);
}

int cq_kv_tree_attend(const cq_kv_geom *g, const cq_kv_tree *t, void *stream) { return tree_attend(g, t, false, stream); }

int cq_selftest_tree_timeout(const cq_kv_geom *g, const cq_kv_tree *t, void *stream) { return tree_attend(g, t, true, stream); }

}  // extern "C"
