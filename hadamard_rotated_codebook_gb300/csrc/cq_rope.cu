// cq_rope.cu -- norms of query and key heads with their position rotation.
//
//   y = x / sqrt(mean(x^2) + eps) * (offset + w);   (y_a, y_b) rotated by t = position * inv_freq[pair]
//
// A head vector is a set of head_dim/2 pairs (a, b). A group of G lanes (a
// power of two, 4 pairs a lane) owns one head: a lane keeps the pairs it
// rotates in registers, so the norm is one shuffle reduction over the group and the
// rotation needs no exchange at all. The pairs of a lane are the same for every
// head, and a warp takes several heads of one token, so each angle is
// computed once per token and warp.
//
// Angles: `rates` are fractions of a turn per position as 64-bit binary
// fractions; position * rate modulo 2^64 is the exact fraction of a turn, whose
// upper 32 bits as a signed number are the angle in [-pi, pi). Rounding that to fp32
// costs 2^-25 of the half turn at any position (a product in fp32 would lose
// all of it at positions of 10^6 and more), without 64-bit floating point,
// which this GPU runs at a small fraction of its fp32 rate.
//
// The bound is memory: each element is read once and written once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "cq_paged.h"

namespace cq {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPairs = 4;  // pairs a lane owns
constexpr int kBatch = 4;  // heads in flight per lane group

struct RopeParams {
    const void *q, *k;
    void *qo, *ko;
    const float *wq, *wk;
    const int32_t *pos;
    int64_t q_st, q_sh, k_st, k_sh, qo_st, qo_sh, ko_st, ko_sh;
    int tokens, hq, heads;  // heads = query + key heads
    int d, rot;
    int q_type, k_type;
    int log_g;              // lanes per head = 1 << log_g
    int chunk, chunks;      // heads per warp task, tasks per token
    float eps, offset, inv_d;
    uint64_t rates[128];
};

template <typename T> struct Vec4;
template <> struct Vec4<float> { using V = float4; };
template <> struct Vec4<__half> { using V = uint2; };
template <> struct Vec4<__nv_bfloat16> { using V = uint2; };

__device__ __forceinline__ void unpack(float4 v, float *x, const float *) {
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
}
__device__ __forceinline__ void unpack(uint2 v, float *x, const __half *) {
    const float2 a = __half22float2(*reinterpret_cast<__half2 *>(&v.x)), b = __half22float2(*reinterpret_cast<__half2 *>(&v.y));
    x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
}
__device__ __forceinline__ void unpack(uint2 v, float *x, const __nv_bfloat16 *) {
    x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xFFFF0000u);
    x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xFFFF0000u);
}
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

__device__ __forceinline__ void store1(void *base, int64_t off, int type, float v) {
    if (type == CQ_T_F32) static_cast<float *>(base)[off] = v;
    else if (type == CQ_T_F16) static_cast<__half *>(base)[off] = __float2half_rn(v);
    else static_cast<__nv_bfloat16 *>(base)[off] = __float2bfloat16_rn(v);
}
__device__ __forceinline__ void store4(void *base, int64_t off, int type, const float *v) {
    if (type == CQ_T_F32) {
        *reinterpret_cast<float4 *>(static_cast<float *>(base) + off) = make_float4(v[0], v[1], v[2], v[3]);
    } else if (type == CQ_T_F16) {
        const __half2 a = __floats2half2_rn(v[0], v[1]), b = __floats2half2_rn(v[2], v[3]);
        *reinterpret_cast<uint2 *>(static_cast<__half *>(base) + off) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    } else {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(base) + off) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    }
}

// Element offsets of the two members of pair p.
__device__ __forceinline__ int2 pair_at(int p, int d, int rot, bool il) {
    if (il) return make_int2(2 * p, 2 * p + 1);
    const int half = rot >> 1;
    if (p < half) return make_int2(p, p + half);
    const int t = p - half;
    return make_int2(rot + t, rot + t + ((d - rot) >> 1));
}

// VEC: every lane's pairs are two aligned runs of four elements (`A` and `B`: of
// adjacent pairs where IL, else of the first and of the second members).
template <typename T, bool IL, bool VEC>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const __grid_constant__ RopeParams p) {
    using V = typename Vec4<T>::V;
    __shared__ uint64_t s_rate[128];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid < 128) s_rate[tid] = tid < (p.rot >> 1) ? p.rates[tid] : 0;  // a pair past rot_dim turns by zero
    __syncthreads();
    const int g = 1 << p.log_g, sub = lane & (g - 1), slot = lane >> p.log_g, slots = 32 >> p.log_g;
    const int p0 = sub * kPairs, half_d = p.d >> 1;
    const bool live = p0 < half_d;
    int at[2 * kPairs];  // element offsets: pair j is at[j], at[kPairs + j] (VEC: at[0] and at[kPairs] start the runs)
    if (VEC && IL) {
        at[0] = 2 * p0, at[kPairs] = 2 * p0 + 4;
    } else if (VEC) {
        const int2 o = pair_at(p0, p.d, p.rot, false);
        at[0] = o.x, at[kPairs] = o.y;
    } else {
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            const int2 o = pair_at(min(p0 + j, half_d - 1), p.d, p.rot, IL);
            at[j] = o.x, at[kPairs + j] = o.y;
        }
    }
    // element offset of register x[i]; registers hold first members, then second ones (VEC && IL: the run itself)
    auto elem = [&](int i) { return VEC ? at[i & kPairs] + (i & (kPairs - 1)) : at[i]; };
    const long long tasks = (long long)p.tokens * p.chunks;
    for (long long task = (long long)blockIdx.x * kWarps + warp; task < tasks; task += (long long)gridDim.x * kWarps) {
        const int t = (int)(task / p.chunks), c = (int)(task - (long long)t * p.chunks);
        float cs[kPairs], sn[kPairs];
        const uint64_t pos = p.rot ? (uint64_t)(int64_t)p.pos[t] : 0;
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            const uint64_t turn = pos * s_rate[min(p0 + j, 127)];
            sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &sn[j], &cs[j]);
        }
        const int h1 = min(p.heads, (c + 1) * p.chunk);
        for (int hb = c * p.chunk; hb < h1; hb += kBatch * slots) {
            float x[kBatch][2 * kPairs];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int h = hb + b * slots + slot;
#pragma unroll
                for (int i = 0; i < 2 * kPairs; ++i) x[b][i] = 0.0f;
                if (h < h1 && live) {
                    const bool is_q = h < p.hq;
                    const T *src = static_cast<const T *>(is_q ? p.q : p.k) +
                                   (is_q ? t * p.q_st + h * p.q_sh : t * p.k_st + (h - p.hq) * p.k_sh);
                    if (VEC) {
                        unpack(*reinterpret_cast<const V *>(src + at[0]), &x[b][0], (const T *)nullptr);
                        unpack(*reinterpret_cast<const V *>(src + at[kPairs]), &x[b][kPairs], (const T *)nullptr);
                    } else {
#pragma unroll
                        for (int j = 0; j < kPairs; ++j)
                            if (p0 + j < half_d) x[b][j] = to_f(src[at[j]]), x[b][kPairs + j] = to_f(src[at[kPairs + j]]);
                    }
                }
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                if (hb + b * slots >= h1) break;  // uniform: the shuffles below take all lanes
                const int h = hb + b * slots + slot;
                float s = 0.0f;
#pragma unroll
                for (int i = 0; i < 2 * kPairs; ++i) s = fmaf(x[b][i], x[b][i], s);
                for (int o = g >> 1; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
                if (h >= h1 || !live) continue;
                const bool is_q = h < p.hq;
                const float inv = rsqrtf(fmaf(s, p.inv_d, p.eps));
                const float *w = is_q ? p.wq : p.wk;
                float y[2 * kPairs];
#pragma unroll
                for (int i = 0; i < 2 * kPairs; ++i) y[i] = x[b][i] * inv * (w ? p.offset + w[elem(i)] : p.offset + 1.0f);
#pragma unroll
                for (int j = 0; j < kPairs; ++j) {
                    const int a = VEC && IL ? 2 * j : j, e = VEC && IL ? 2 * j + 1 : kPairs + j;
                    const float u = y[a], v = y[e];
                    y[a] = u * cs[j] - v * sn[j];
                    y[e] = v * cs[j] + u * sn[j];
                }
                void *dst = is_q ? p.qo : p.ko;
                const int type = is_q ? p.q_type : p.k_type;
                const int64_t base = is_q ? t * p.qo_st + h * p.qo_sh : t * p.ko_st + (h - p.hq) * p.ko_sh;
                if (VEC) {
                    store4(dst, base + at[0], type, &y[0]);
                    store4(dst, base + at[kPairs], type, &y[kPairs]);
                } else {
#pragma unroll
                    for (int j = 0; j < kPairs; ++j)
                        if (p0 + j < half_d) {
                            store1(dst, base + at[j], type, y[j]);
                            store1(dst, base + at[kPairs + j], type, y[kPairs + j]);
                        }
                }
            }
        }
    }
}

int size_of(int type) { return type == CQ_T_F32 ? 4 : 2; }

template <typename T>
void launch_t(const RopeParams &p, bool il, bool vec, int grid, cudaStream_t st) {
    if (il && vec) qk_norm_rope_kernel<T, true, true><<<grid, kThreads, 0, st>>>(p);
    else if (il) qk_norm_rope_kernel<T, true, false><<<grid, kThreads, 0, st>>>(p);
    else if (vec) qk_norm_rope_kernel<T, false, true><<<grid, kThreads, 0, st>>>(p);
    else qk_norm_rope_kernel<T, false, false><<<grid, kThreads, 0, st>>>(p);
}

}  // namespace

int launch_qk_norm_rope(const cq_qk_desc &d, void *stream) {
    RopeParams p;
    p.q = d.q, p.k = d.k, p.qo = d.q_out, p.ko = d.k_out;
    p.wq = d.q_weight, p.wk = d.k_weight;
    p.pos = d.positions;
    p.q_st = d.q_stride_t, p.q_sh = d.q_stride_h, p.k_st = d.k_stride_t, p.k_sh = d.k_stride_h;
    p.qo_st = d.qo_stride_t, p.qo_sh = d.qo_stride_h, p.ko_st = d.ko_stride_t, p.ko_sh = d.ko_stride_h;
    p.tokens = d.n_tokens, p.hq = d.n_q_heads, p.heads = d.n_q_heads + d.n_kv_heads;
    p.d = d.head_dim, p.rot = d.rot_dim;
    p.q_type = d.q_out_dtype, p.k_type = d.k_out_dtype;
    p.eps = d.eps, p.offset = d.weight_offset, p.inv_d = 1.0f / (float)d.head_dim;
    for (int i = 0; i < d.rot_dim / 2; ++i) p.rates[i] = d.rates[i];
    const int lanes = (d.head_dim / 2 + kPairs - 1) / kPairs;
    p.log_g = 0;
    while ((1 << p.log_g) < lanes) ++p.log_g;
    // Runs of four elements need every offset of a run to be a multiple of four.
    const bool il = d.interleaved != 0;
    bool vec = il ? d.head_dim % 8 == 0 : (d.rot_dim / 2) % 4 == 0 && (d.head_dim - d.rot_dim) / 2 % 4 == 0;
    auto runs = [&](const void *b, int64_t st, int64_t sh, int type, int heads) {
        vec = vec && (!heads || ((reinterpret_cast<uintptr_t>(b) % (4 * size_of(type)) == 0) && st % 4 == 0 && sh % 4 == 0));
    };
    runs(p.q, p.q_st, p.q_sh, d.in_dtype, d.n_q_heads);
    runs(p.k, p.k_st, p.k_sh, d.in_dtype, d.n_kv_heads);
    runs(p.qo, p.qo_st, p.qo_sh, p.q_type, d.n_q_heads);
    runs(p.ko, p.ko_st, p.ko_sh, p.k_type, d.n_kv_heads);
    // A warp takes as many of a token's heads as still leave every SM 32 warps.
    const int slots = 32 >> p.log_g, sms = sm_count();
    p.chunk = slots;
    while (p.chunk < p.heads && (long long)p.tokens * ((p.heads + 2 * p.chunk - 1) / (2 * p.chunk)) >= 32LL * sms) p.chunk *= 2;
    p.chunks = (p.heads + p.chunk - 1) / p.chunk;
    const long long blocks = ((long long)p.tokens * p.chunks + kWarps - 1) / kWarps;
    const int grid = (int)std::min<long long>(blocks, 8LL * sms);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (d.in_dtype == CQ_T_F32) launch_t<float>(p, il, vec, grid, st);
    else if (d.in_dtype == CQ_T_F16) launch_t<__half>(p, il, vec, grid, st);
    else launch_t<__nv_bfloat16>(p, il, vec, grid, st);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return set_error(CQ_ERR_CUDA, "norm and rotation launch: %s", cudaGetErrorString(e));
    return CQ_OK;
}

}  // namespace cq
