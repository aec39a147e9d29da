// cq_layer_host.cpp -- host side of the block norm's and the adapters' entry points: argument checks, alignment.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "cq_layer.h"

using namespace cq;

namespace {

constexpr int kMaxSide = 1 << 28;  // inputs and outputs of an adapted projection

bool is_float(int type) { return type >= CQ_T_F32 && type <= CQ_T_BF16; }
bool aligned(const void *p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// Rows of a tensor: n of them, `bytes` long and `stride` bytes apart.
struct Rows {
    const void *at;
    int64_t stride, bytes;
    int type;  // of the elements
};
Rows rows_of(const void *at, int64_t stride, int64_t width, int type) {
    const int size = type == CQ_T_F32 ? 4 : type == CQ_T_I8 ? 1 : 2;
    return {at, stride * size, width * size, type};
}
// a / b of whole numbers, rounded down; b above zero.
__int128 floor_div(__int128 a, __int128 b) { return a / b - (a % b < 0); }
// Whether two tensors of n rows share a byte. (Column slices of one tensor do not, though one's rows lie between the other's.)
bool overlap(Rows a, Rows b, int64_t n) {
    if (!a.at || !b.at || n < 1 || a.bytes < 1 || b.bytes < 1) return false;
    if (n == 1) a.stride = b.stride = 0;
    __int128 p = reinterpret_cast<uintptr_t>(a.at), q = reinterpret_cast<uintptr_t>(b.at), s = a.stride, t = b.stride;
    if (s < 0) p += s * (n - 1), s = -s;  // the last row first
    if (t < 0) q += t * (n - 1), t = -t;
    if (p >= q + t * (n - 1) + b.bytes || q >= p + s * (n - 1) + a.bytes) return false;
    // Rows of b, `step` apart and numbered lo .. hi, of which one meets `bytes` from `at` on.
    auto meets = [&](__int128 at, int64_t bytes, __int128 step, int64_t lo, int64_t hi) {
        if (step == 0) return at < q + b.bytes && q < at + bytes;
        const __int128 first = floor_div(at - b.bytes - q, step) + 1, last = floor_div(at + bytes - 1 - q, step);
        return std::max<__int128>(first, lo) <= std::min<__int128>(last, hi);
    };
    if (s == t) return meets(p, a.bytes, s, 1 - n, n - 1);  // only the distance of the rows' numbers counts
    for (int64_t i = 0; i < n; ++i)
        if (meets(p + s * i, a.bytes, t, 0, n - 1)) return true;
    return false;
}
// The same tensor, element by element.
bool same(const Rows &a, const Rows &b, int64_t n) { return a.at == b.at && a.type == b.type && (n == 1 || a.stride == b.stride); }

// How a call is cut up, apart from its alignment; the workspace's bytes, or 0.
size_t lora_plan(const cq_lora_desc &d, bool few, bool tensor, LoraParams &p) {
    const int tiles = lora_rank_tiles(d.rank), ranks = 16 * tiles, tok = lora_tokens(d.x_dtype, tiles, few, tensor);
    const long long pieces = std::min<long long>(d.n_tokens, (long long)d.n_seqs + d.n_tokens / tok);
    p.few = few;
    p.tensor = tensor;
    p.u_row = (d.rank + ranks - 1) / ranks * ranks;
    // Parts of k, while a block keeps 512 inputs and more: no more blocks than run at once (three an SM for few tokens: 32 requests of 8
    // tokens 11.0 us, 13.3 with twice the parts; two on tcgen05: 8190 tokens, rank 64 73 us, 77 with twice), as the sums of all are
    // read again. fp32 prompts, which cost more instructions, want the last round full (50.2 us, 51.7 with half the parts).
    const long long room = tensor ? sm_count() : few ? 3ll * sm_count() / 2 : 3ll * sm_count() - 1;
    p.splits = 1;
    while (p.splits < kMaxSplits && pieces * d.n_mats * p.splits <= room && d.in >= 1024 * p.splits) p.splits *= 2;
    p.runs = 1;
    if (pieces * p.splits > INT_MAX) {
        set_error(CQ_ERR_SHAPE, "%d tokens of %d requests are too many for one call", d.n_tokens, d.n_seqs);
        return 0;
    }
    p.pieces = (int)pieces;
    return (size_t)d.n_mats * p.splits * d.n_tokens * p.u_row * sizeof(float);
}
// Pieces of 8 tokens on mma.sync: where requests have few tokens each, whose adapters are then what there is to read, and where there
// are few tokens in all, as tcgen05's kernels take 6 us longer to begin and end. Their cost a token goes by the ranks and, as y is
// read and written, more by the outputs than by the inputs. (4096 to 4096, int8, few against many: rank 16, a prompt of 40 tokens 5.5 us
// against 12.5, of 512 11.8 against 15.4, of 1024 18.0 against 18.4, four of 512 30 against 24; 32 requests of 20 15 against 25; rank 64,
// one of 512 23.4 against 19.7, 16 requests of 32 29 against 24, 64 of 16 50 against 49.)
// The rule knows a call's sums alone, and takes the slower kernels in between: 16 requests of 48 tokens at rank 16 (21 us, 15 with few), 32
// of 50 (32, 28), at rank 64 one of 256 (18, 14) and 8 of 28 (20, 16). It counts rows that no request covers, so that 64 decodes in
// buffers of 4096 rows take the kernels of many tokens (92 us, 26 with few), and it does not see one prompt of 2000 tokens beside 255
// single tokens (rank 64: 145 us, 82 and 29 in calls of their own; rank 16: 51, 25 and 24).
bool lora_few(const cq_lora_desc &d) {
    const long long tiles = (d.rank + 15) / 16;
    long long side = d.in;
    for (int j = 0; j < d.n_mats; ++j) side += 3ll * d.out[j];
    return d.n_tokens <= std::max(16ll, 32 / tiles) * d.n_seqs || (double)d.n_tokens * (double)(tiles * side) <= 12e6;
}

}  // namespace

extern "C" {

static int block_norm(const cq_norm_desc *d, bool give_up, void *stream) {
    clear_error();
    if (!d) return set_error(CQ_ERR_ARG, "null descriptor");
    if (!is_float(d->x_dtype) || !is_float(d->residual_dtype) || (!is_float(d->out_dtype) && d->out_dtype != CQ_T_I8))
        return set_error(CQ_ERR_ARG, "unknown element types %d, %d, %d", d->x_dtype, d->residual_dtype, d->out_dtype);
    if (d->n_tokens < 0) return set_error(CQ_ERR_SHAPE, "negative size");
    if (d->width < 1 || d->width > CQ_NORM_MAX_WIDTH)
        return set_error(CQ_ERR_SHAPE, "width must be 1..%d, got %d", CQ_NORM_MAX_WIDTH, d->width);
    if (d->gate && d->gate_width != 1 && d->gate_width != d->width)
        return set_error(CQ_ERR_SHAPE, "a gate has 1 or %d elements a token, got %d", d->width, d->gate_width);
    if (d->gate_act < CQ_GATE_PLAIN || d->gate_act > CQ_GATE_SILU) return set_error(CQ_ERR_ARG, "unknown gate function %d", d->gate_act);
    if (!(d->eps >= 0) || !std::isfinite(d->eps) || !std::isfinite(d->weight_offset) || !std::isfinite(d->branch_scale) ||
        !std::isfinite(d->residual_scale))
        return set_error(CQ_ERR_ARG, "eps must be finite and not negative, weight_offset and the scales finite");
    if (d->n_tokens == 0) return CQ_OK;
    if (!d->x || !d->out) return set_error(CQ_ERR_ARG, "null x or out");
    if (d->out_dtype == CQ_T_I8 && !d->out_scale) return set_error(CQ_ERR_ARG, "int8 outputs need out_scale");
    if (d->n_tokens > 1 && ((d->residual_out && d->residual_out_stride < d->width) || d->out_stride < d->width))
        return set_error(CQ_ERR_SHAPE, "output rows of %d elements are %lld and %lld apart", d->width, (long long)d->residual_out_stride,
                         (long long)d->out_stride);
    // An element of an output may take the place of the same element of an input: the lane that writes it has read it. Anything else would be
    // written while others read.
    const int64_t n = d->n_tokens, w = d->width;
    const Rows out[3] = {rows_of(d->out, d->out_stride, w, d->out_dtype), rows_of(d->residual_out, d->residual_out_stride, w, d->residual_dtype),
                         rows_of(d->out_dtype == CQ_T_I8 ? d->out_scale : nullptr, 1, 1, CQ_T_F32)};
    const Rows in[5] = {rows_of(d->x, d->x_stride, w, d->x_dtype), rows_of(d->residual, d->residual_stride, w, d->residual_dtype),
                        rows_of(d->gate, d->gate_stride, d->gate_width, d->x_dtype), rows_of(d->weight, 0, w, CQ_T_F32),
                        rows_of(d->branch_weight, 0, w, CQ_T_F32)};
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j], n)) return set_error(CQ_ERR_ARG, "two outputs share memory");
        for (int j = 0; j < 5; ++j)
            if (overlap(out[i], in[j], n) && !(i < 2 && j < 3 && out[i].bytes == in[j].bytes && same(out[i], in[j], n)))
                return set_error(CQ_ERR_ARG, "an output and an input share memory in another way than element by element");
    }
    return launch_block_norm(*d, give_up, stream);
}

int cq_block_norm(const cq_norm_desc *d, void *stream) { return block_norm(d, false, stream); }
int cq_selftest_norm_timeout(const cq_norm_desc *d, void *stream) { return block_norm(d, true, stream); }

// Sizes and types that a call needs right, whatever its pointers.
static int check_lora(const cq_lora_desc *d) {
    if (!d) return set_error(CQ_ERR_ARG, "null descriptor");
    if (d->w_dtype != CQ_T_F16 && d->w_dtype != CQ_T_BF16) return set_error(CQ_ERR_ARG, "weights are fp16 or bf16, got element type %d", d->w_dtype);
    if (d->x_dtype != CQ_T_F32 && d->x_dtype != CQ_T_I8 && d->x_dtype != d->w_dtype)
        return set_error(CQ_ERR_ARG, "activations are fp32, int8 or of the weights' type, got element type %d", d->x_dtype);
    if (d->n_mats < 0 || d->n_mats > CQ_LORA_MAX_MATS)
        return set_error(CQ_ERR_SHAPE, "at most %d matrices, got %d", CQ_LORA_MAX_MATS, d->n_mats);
    if (d->n_tokens < 0 || d->n_seqs < 0 || d->n_adapters < 0) return set_error(CQ_ERR_SHAPE, "negative size");
    if (d->rank > 0 && d->n_adapters > INT_MAX / d->rank) return set_error(CQ_ERR_SHAPE, "%d adapters of rank %d are too many", d->n_adapters, d->rank);
    if (d->in < 1 || d->in > kMaxSide) return set_error(CQ_ERR_SHAPE, "in must be 1..%d, got %d", kMaxSide, d->in);
    if (d->rank < 1 || d->rank > CQ_LORA_MAX_RANK) return set_error(CQ_ERR_SHAPE, "rank must be 1..%d, got %d", CQ_LORA_MAX_RANK, d->rank);
    for (int j = 0; j < d->n_mats; ++j)
        if (d->out[j] < 1 || d->out[j] > kMaxSide) return set_error(CQ_ERR_SHAPE, "out must be 1..%d, got %d", kMaxSide, d->out[j]);
    return CQ_OK;
}

size_t cq_lora_workspace(const cq_lora_desc *d) {
    clear_error();
    LoraParams p;
    if (check_lora(d) || !d->n_mats || !d->n_tokens || !d->n_seqs) return 0;
    const size_t plain = lora_plan(*d, false, false, p), many = lora_plan(*d, false, true, p), few = lora_plan(*d, true, false, p);
    return plain && many && few ? std::max(plain, std::max(many, few)) : 0;
}

static int lora_add(const cq_lora_desc *d, bool give_up, void *stream) {
    clear_error();
    const int st = check_lora(d);
    if (st) return st;
    if (d->n_mats == 0 || d->n_tokens == 0 || d->n_seqs == 0) return CQ_OK;
    if (!d->x || !d->adapters || !d->cu_tokens) return set_error(CQ_ERR_ARG, "null x, adapters or cu_tokens");
    if (d->x_dtype == CQ_T_I8 && !d->x_scale) return set_error(CQ_ERR_ARG, "int8 activations need x_scale");
    for (int j = 0; j < d->n_mats; ++j) {
        if (!d->y[j] || !d->y_out[j]) return set_error(CQ_ERR_ARG, "null y");
        if (d->n_adapters && (!d->a[j] || !d->b[j])) return set_error(CQ_ERR_ARG, "null a or b");
        if (d->n_tokens > 1 && d->y_out_stride[j] < d->out[j])
            return set_error(CQ_ERR_SHAPE, "output rows of %d elements are %lld apart", d->out[j], (long long)d->y_out_stride[j]);
        if (d->y[j] == d->y_out[j] && d->n_tokens > 1 && d->y_stride[j] != d->y_out_stride[j])
            return set_error(CQ_ERR_SHAPE, "y is added to in place with rows %lld and %lld apart", (long long)d->y_stride[j],
                             (long long)d->y_out_stride[j]);
    }
    const Rows x = rows_of(d->x, d->x_stride, d->in, d->x_dtype);
    for (int j = 0; j < d->n_mats; ++j) {
        const Rows o = rows_of(d->y_out[j], d->y_out_stride[j], d->out[j], CQ_T_F32);
        if (overlap(o, x, d->n_tokens)) return set_error(CQ_ERR_ARG, "an output shares memory with x");
        for (int k = 0; k < d->n_mats; ++k) {
            const Rows y = rows_of(d->y[k], d->y_stride[k], d->out[k], CQ_T_F32);
            if ((k != j && overlap(o, rows_of(d->y_out[k], d->y_out_stride[k], d->out[k], CQ_T_F32), d->n_tokens)) ||
                (!(k == j && same(o, y, d->n_tokens)) && overlap(o, y, d->n_tokens)))
                return set_error(CQ_ERR_ARG, "output %d shares memory with output %d or its y", j, k);
        }
    }
    LoraParams p;
    p.d = *d;
    // Where 16-byte loads (8 of int8) and 16-byte accesses to y may be used; single elements elsewhere.
    const int size = d->x_dtype == CQ_T_F32 ? 4 : d->x_dtype == CQ_T_I8 ? 1 : 2, run = d->x_dtype == CQ_T_I8 ? 8 : 16;
    p.vec = d->in % 8 == 0 && d->n_adapters && aligned(d->x, run) && (d->n_tokens == 1 || d->x_stride * size % run == 0);
    p.vec_b = d->rank % 4 == 0;
    for (int j = 0; j < d->n_mats; ++j) {
        p.vec = p.vec && aligned(d->a[j], 16);
        p.vec_b = p.vec_b && aligned(d->b[j], 8);
        p.vec_y[j] = d->out[j] % 4 == 0 && aligned(d->y[j], 16) && aligned(d->y_out[j], 16) &&
                     (d->n_tokens == 1 || (d->y_stride[j] % 4 == 0 && d->y_stride[j] >= d->out[j] && d->y_out_stride[j] % 4 == 0));
    }
    const bool few = p.vec && lora_few(*d);
    const bool tensor = !few && p.vec && d->x_dtype != CQ_T_F32 && aligned(d->x, 16) && (d->n_tokens == 1 || (d->x_stride * size % 16 == 0 && d->x_stride >= d->in));
    const size_t need = lora_plan(*d, few, tensor, p);
    if (!need) return CQ_ERR_SHAPE;
    if (!d->workspace || d->workspace_bytes < need || !aligned(d->workspace, 16))
        return set_error(CQ_ERR_ARG, "workspace of %zu bytes needed (16-byte aligned), got %zu", need, d->workspace ? d->workspace_bytes : 0);
    p.u = static_cast<float *>(d->workspace);
    p.status = device_status_ptr();
    p.give_up = give_up;
    if (!p.status) return set_error(CQ_ERR_CUDA, "no device status word");
    return d->w_dtype == CQ_T_F16 ? launch_lora_f16(p, stream) : launch_lora_bf16(p, stream);
}

int cq_lora_add(const cq_lora_desc *d, void *stream) { return lora_add(d, false, stream); }
int cq_selftest_lora_timeout(const cq_lora_desc *d, void *stream) { return lora_add(d, true, stream); }

}  // extern "C"
