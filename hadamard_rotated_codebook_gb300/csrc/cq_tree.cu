// cq_tree.cu -- attention of drafted tokens over a paged CQ cache.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>

#include "cq_paged.h"

namespace cq {
namespace {

constexpr int kThreads = 128;

struct TreeParams {
    cq_kv_tree t;
    TreeUnit unit[kMaxUnits];
    unsigned int *status;
    float lk[16], lv[16];
    int n_units, hq, hkv, dk, dv, wk, wv, kgroups, vgroups;
    float scale;
};

__device__ __forceinline__ int code_at(const uint8_t *row, int k, int w) {
    const int bit = k * w;
    unsigned v = row[bit >> 3];
    if ((bit & 7) + w > 8) v |= row[(bit >> 3) + 1] << 8;
    return v >> (bit & 7) & ((1 << w) - 1);
}

__device__ void fwht128(float *z, int tid) {
    for (int h = 1; h < 128; h <<= 1) {
        __syncthreads();
        float v = 0.0f;
        const float a = z[tid], b = z[tid ^ h];
        v = (tid & h) ? b - a : a + b;
        __syncthreads();
        z[tid] = v;
    }
    __syncthreads();
}

__device__ float block_reduce(float v, bool mx, float *buf, int tid) {
    __syncthreads();
    buf[tid] = v;
    __syncthreads();
    for (int h = 64; h; h >>= 1) {
        if (tid < h) buf[tid] = mx ? fmaxf(buf[tid], buf[tid + h]) : buf[tid] + buf[tid + h];
        __syncthreads();
    }
    return buf[0];
}

// One request as the kernel takes it: lengths outside the given sizes are cut to
// them (`bad`), so that no index leaves its buffer whatever the device holds.
struct Seq {
    int first, n, ctx, len;
    bool bad;
};
__device__ __forceinline__ Seq seq_at(const TreeParams &p, int s) {
    Seq q;
    const int a = p.t.cu_nodes[s], b = p.t.cu_nodes[s + 1];
    q.first = a;
    q.bad = a < 0 || b < a || b > p.t.n_nodes;
    q.n = q.bad ? 0 : min(b - a, p.t.max_nodes);
    q.bad |= !q.bad && b - a > p.t.max_nodes;
    const long long room = min((long long)p.t.max_blocks * p.t.block_size, (long long)INT_MAX);
    long long ctx = p.t.context_lens[s];
    if (ctx < 0) q.bad = true, ctx = 0;
    q.bad |= q.n && ctx + q.n > room;
    q.ctx = (int)ctx;
    q.len = q.n ? (int)min(ctx + q.n, room) : 0;
    return q;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) tree_kernel(const __grid_constant__ TreeParams p) {
    __shared__ float z[2][128], buf[128], pr[128];
    __shared__ int rows[128];
    const int tid = threadIdx.x, node = blockIdx.x, head = blockIdx.y;
    if (node == 0 && head == 0)
        for (int s = tid; s < p.t.n_seqs; s += kThreads)
            if (seq_at(p, s).bad) atomicOr(p.status, kStatusIndex);
    int s = 0;
    while (s + 1 < p.t.n_seqs && p.t.cu_nodes[s + 1] <= node) ++s;
    const Seq q0 = seq_at(p, s);
    const int i = node - q0.first, ctx = q0.ctx, len = q0.len, h = head / (p.hq / p.hkv);
    if (i < 0 || i >= q0.n) return;
    const int k0 = h * p.dk, gk = k0 / 128, ngk = (k0 + p.dk + 127) / 128 - gk;
    const int v0 = h * p.dv, gv = v0 / 128, ngv = (v0 + p.dv + 127) / 128 - gv;
    const T *q = static_cast<const T *>(p.t.q) + node * p.t.q_stride_t + head * p.t.q_stride_h;
    for (int g = 0; g < ngk; ++g) {
        const int d = (gk + g) * 128 + tid - k0;
        z[g][tid] = d >= 0 && d < p.dk ? (float)q[d] : 0.0f;
        fwht128(z[g], tid);
    }
    const size_t krow = (size_t)p.kgroups * 16 * p.wk, vrow = (size_t)p.vgroups * 16 * p.wv;
    const __half *kn = reinterpret_cast<const __half *>(p.t.k_cache + p.t.cap * krow);
    const __half *vn = reinterpret_cast<const __half *>(p.t.v_cache + p.t.cap * vrow);
    float m = -INFINITY, l = 0.0f, acc[2] = {0.0f, 0.0f};
    for (int base = 0; base < len; base += 128) {
        const int t = base + tid, j = t - ctx;
        bool see = t < len;
        if (see && j >= 0) see = p.t.mask ? p.t.mask[(size_t)node * p.t.mask_words + (j >> 5)] >> (j & 31) & 1 : j <= i;
        long long row = -1;
        if (see) {
            const int b = t / p.t.block_size;
            const int blk = b < p.t.max_blocks ? p.t.block_table[s * p.t.table_stride + b] : -1;
            row = (long long)blk * p.t.block_size + t % p.t.block_size;
            if (blk < 0 || row >= p.t.cap) {
                see = false;
                atomicOr(p.status, kStatusIndex);
            }
        }
        float x = -INFINITY;
        if (see) {
            x = 0.0f;
            for (int g = 0; g < ngk; ++g) {
                const uint8_t *c = p.t.k_cache + row * krow + (size_t)(gk + g) * 16 * p.wk;
                float dot = 0.0f;
                for (int k = 0; k < 128; ++k) dot += z[g][k] * p.lk[code_at(c, k, p.wk)];
                x += dot * __half2float(kn[row * p.kgroups + gk + g]);
            }
            x *= p.scale * 0.08838834764831845f;
        }
        const float mt = fmaxf(m, block_reduce(x, true, buf, tid));
        const float e = see ? expf(x - mt) : 0.0f;
        const float f = m == -INFINITY ? 0.0f : expf(m - mt);
        l = l * f + block_reduce(e, false, buf, tid);
        acc[0] *= f, acc[1] *= f;
        m = mt;
        pr[tid] = e;
        rows[tid] = see ? (int)row : -1;
        __syncthreads();
        for (int u = 0; u < 128 && base + u < len; ++u) {
            if (rows[u] < 0) continue;
            const long long r = rows[u];
            for (int g = 0; g < ngv; ++g)
                acc[g] += pr[u] * __half2float(vn[r * p.vgroups + gv + g]) *
                          p.lv[code_at(p.t.v_cache + r * vrow + (size_t)(gv + g) * 16 * p.wv, tid, p.wv)];
        }
        __syncthreads();
    }
    for (int g = 0; g < ngv; ++g) {
        z[g][tid] = l > 0.0f || l != l ? acc[g] / l * 0.08838834764831845f : 0.0f;
        fwht128(z[g], tid);
    }
    T *o = static_cast<T *>(p.t.o) + node * p.t.o_stride_t + head * p.t.o_stride_h;
    for (int d = tid; d < p.dv; d += 128) {
        const int c = v0 + d - gv * 128;
        o[d] = (T)z[c >> 7][c & 127];
    }
}

}  // namespace

size_t tree_workspace(const cq_kv_geom &, int, int) { return 0; }

int launch_kv_tree_attend(const cq_kv_geom &g, const cq_kv_tree &t, const float *lk, const float *lv, void *stream) {
    TreeParams p;
    p.t = t;
    p.n_units = tree_units(g, p.unit);
    p.hq = g.n_q_heads, p.hkv = g.n_kv_heads, p.dk = g.head_dim_k, p.dv = g.head_dim_v;
    p.wk = width_of(g.k_bits), p.wv = width_of(g.v_bits);
    p.kgroups = in_padded(p.hkv * p.dk) / kGroup, p.vgroups = in_padded(p.hkv * p.dv) / kGroup;
    p.scale = g.scale;
    p.status = device_status_ptr();
    if (!p.status) return set_error(CQ_ERR_CUDA, "no device status word");
    std::copy(lk, lk + 16, p.lk);
    std::copy(lv, lv + 16, p.lv);
    const dim3 grid(t.n_nodes, g.n_q_heads);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (t.dtype == CQ_T_F16) tree_kernel<__half><<<grid, kThreads, 0, st>>>(p);
    else tree_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return set_error(CQ_ERR_CUDA, "tree attention launch: %s", cudaGetErrorString(e));
    return CQ_OK;
}

}  // namespace cq
