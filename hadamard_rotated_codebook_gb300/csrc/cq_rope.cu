// cq_rope.cu -- norms of query and key heads with their position rotation.
//
//   y = x / sqrt(mean(x^2) + eps) * (offset + w);   (y_a, y_b) rotated by t = position * inv_freq[pair]
//
// A head vector is a set of head_dim/2 pairs (a, b). A group of G lanes (a
// power of two; a lane has 4 pairs, or 8 of a 16-bit type: 16-byte loads) owns one head: a lane keeps the pairs it
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
// The bound is memory: each element is read once and written once. 16383 tokens of 40 heads of 128 in bf16 (335 MB) take
// 63.7 us, 5.3 TB/s or 78% of the copy rate; issue slots are used to two thirds and the shared-memory pipe (weights, staging of
// loads and stores) to about half, with 24 warps on an SM. Small steps are a launch: 13 to 18 us through the Python
// binding, whose calls are what they cost: the kernel itself takes 5 to 6 from cold caches.
// Tried and no faster: loads a batch of heads ahead (63.9 us), 4 blocks of 64 registers (66 to 83 us).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "cq_paged.h"

namespace cq {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBatch = 4;   // heads in flight per lane group
constexpr int kBlocks = 3;  // resident per SM, and launched: more than one wave costs 2.5 us of 67

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

// N consecutive elements as registers: N * sizeof(T) bytes, 8 or 16.
template <int BYTES> struct Raw;
template <> struct Raw<8> { using V = uint2; };
template <> struct Raw<16> { using V = uint4; };
__device__ __forceinline__ float to_f32(uint32_t v, int half, const __half *) {
    return __half2float(__ushort_as_half((unsigned short)(half ? v >> 16 : v)));
}
__device__ __forceinline__ float to_f32(uint32_t v, int half, const __nv_bfloat16 *) { return __uint_as_float(half ? v & 0xFFFF0000u : v << 16); }
__device__ __forceinline__ float to_f32(uint32_t v, int, const float *) { return __uint_as_float(v); }
template <typename T, int N, typename V>
__device__ __forceinline__ void unpack(const V &v, float *x) {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(&v);
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] = sizeof(T) == 4 ? to_f32(w[j], 0, (const T *)nullptr) : to_f32(w[j / 2], j & 1, (const T *)nullptr);
}
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

__device__ __forceinline__ void store1(void *base, int64_t off, int type, float v) {
    if (type == CQ_T_F32) static_cast<float *>(base)[off] = v;
    else if (type == CQ_T_F16) static_cast<__half *>(base)[off] = __float2half_rn(v);
    else static_cast<__nv_bfloat16 *>(base)[off] = __float2bfloat16_rn(v);
}
// N consecutive elements, N * size bytes a multiple of 8.
template <int N>
__device__ __forceinline__ void store_run(void *base, int64_t off, int type, const float *v) {
    if (type == CQ_T_F32) {
#pragma unroll
        for (int j = 0; j < N; j += 4) __stcs(reinterpret_cast<float4 *>(static_cast<float *>(base) + off + j), make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]));
        return;
    }
    uint32_t w[N / 2];
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
        if (type == CQ_T_F16) {
            const __half2 a = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
            w[j] = *reinterpret_cast<const uint32_t *>(&a);
        } else {
            const __nv_bfloat162 a = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
            w[j] = *reinterpret_cast<const uint32_t *>(&a);
        }
    }
    uint16_t *dst = static_cast<uint16_t *>(base) + off;
    if (N == 8) __stcs(reinterpret_cast<uint4 *>(dst), make_uint4(w[0], w[1], w[N / 2 - 2], w[N / 2 - 1]));
    else __stcs(reinterpret_cast<uint2 *>(dst), make_uint2(w[0], w[1]));
}

// Element offsets of the two members of pair p.
__device__ __forceinline__ int2 pair_at(int p, int d, int rot, bool il) {
    if (il) return make_int2(2 * p, 2 * p + 1);
    const int half = rot >> 1;
    if (p < half) return make_int2(p, p + half);
    const int t = p - half;
    return make_int2(rot + t, rot + t + ((d - rot) >> 1));
}

// Where the weight of element e lies in shared memory. Runs of 8 are cut in two halves 128 floats apart, so that neighbouring
// lanes' 16-byte loads are neighbours too (in their own order they met in the banks two by two: 67.6 against 66.8 us).
template <int RUN>
__device__ __forceinline__ int weight_at(int e) {
    return RUN == 8 ? (e >> 3 << 2) + (e & 3) + ((e & 4) << 5) : e;
}

// P pairs a lane. VEC: they are two aligned runs of P elements (`A` and `B`: of adjacent pairs where IL, else of the first and
// of the second members).
template <typename T, int P, bool IL, bool VEC>
__global__ void __launch_bounds__(kThreads, kBlocks) qk_norm_rope_kernel(const __grid_constant__ RopeParams p) {
    using V = typename Raw<VEC ? P * (int)sizeof(T) : 16>::V;
    __shared__ uint64_t s_rate[128];
    __shared__ __align__(16) float s_w[2][256];  // offset + weight of queries and keys
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid < 128) s_rate[tid] = tid < (p.rot >> 1) ? p.rates[tid] : 0;  // a pair past rot_dim turns by zero
    for (int i = tid; i < 2 * p.d; i += kThreads) {
        const int k = i >= p.d, e = i - k * p.d;
        const float *w = k ? p.wk : p.wq;
        s_w[k][weight_at<VEC ? P : 1>(e)] = p.offset + (w ? w[e] : 1.0f);
    }
    __syncthreads();
    const int g = 1 << p.log_g, sub = lane & (g - 1), slot = lane >> p.log_g, slots = 32 >> p.log_g;
    const int p0 = sub * P, half_d = p.d >> 1;
    const bool live = p0 < half_d;
    int at[2 * P];  // element offsets: pair j is at[j], at[P + j] (VEC: at[0] and at[P] start the runs)
    if (VEC && IL) {
        at[0] = 2 * p0, at[P] = 2 * p0 + P;
    } else if (VEC) {
        const int2 o = pair_at(min(p0, half_d - P), p.d, p.rot, false);
        at[0] = o.x, at[P] = o.y;
    } else {
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const int2 o = pair_at(min(p0 + j, half_d - 1), p.d, p.rot, IL);
            at[j] = o.x, at[P + j] = o.y;
        }
    }
    // registers hold first members, then second ones (VEC && IL: the run itself)
    const long long tasks = (long long)p.tokens * p.chunks;
    for (long long task = (long long)blockIdx.x * kWarps + warp; task < tasks; task += (long long)gridDim.x * kWarps) {
        const int t = (int)(task / p.chunks), c = (int)(task - (long long)t * p.chunks);
        const int h1 = min(p.heads, (c + 1) * p.chunk);
        float cs[P], sn[P];
        const uint64_t pos = p.rot ? (uint64_t)(int64_t)p.pos[t] : 0;
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const uint64_t turn = pos * s_rate[min(p0 + j, 127)];
            sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &sn[j], &cs[j]);
        }
        for (int hb = c * p.chunk; hb < h1; hb += kBatch * slots) {
            V raw[kBatch][2];
            float x[2 * P];
            auto source = [&](int h) {
                const bool is_q = h < p.hq;
                return static_cast<const T *>(is_q ? p.q : p.k) + (is_q ? t * p.q_st + h * p.q_sh : t * p.k_st + (h - p.hq) * p.k_sh);
            };
            if (VEC) {
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                    const int h = hb + b * slots + slot;
                    raw[b][0] = raw[b][1] = V{};
                    if (h < h1 && live) {
                        const T *src = source(h);
                        raw[b][0] = __ldcs(reinterpret_cast<const V *>(src + at[0]));
                        raw[b][1] = __ldcs(reinterpret_cast<const V *>(src + at[P]));
                    }
                }
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                if (hb + b * slots >= h1) break;  // uniform: the shuffles below take all lanes
                const int h = hb + b * slots + slot;
                if (VEC) {
                    unpack<T, P>(raw[b][0], &x[0]);
                    unpack<T, P>(raw[b][1], &x[P]);
                } else {
#pragma unroll
                    for (int i = 0; i < 2 * P; ++i) x[i] = 0.0f;
                    if (h < h1 && live) {
                        const T *src = source(h);
#pragma unroll
                        for (int j = 0; j < P; ++j)
                            if (p0 + j < half_d) x[j] = to_f(src[at[j]]), x[P + j] = to_f(src[at[P + j]]);
                    }
                }
                // squares pair by pair, four pairs to a partial sum, neighbours first: the same bits for every P and layout
                float part[P / 4];
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const int m = VEC && IL ? 2 * j : j, e = VEC && IL ? 2 * j + 1 : P + j;
                    part[j / 4] = fmaf(x[e], x[e], fmaf(x[m], x[m], j % 4 ? part[j / 4] : 0.0f));
                }
                float s = part[0];
                if (P == 8) s += part[P / 4 - 1];
                for (int o = 1; o < g; o <<= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
                if (h >= h1 || !live) continue;
                const bool is_q = h < p.hq;
                const float inv = rsqrtf(fmaf(s, p.inv_d, p.eps));
                const float *w = s_w[!is_q];
#pragma unroll
                for (int i = 0; i < 2 * P; ++i) x[i] = x[i] * inv * w[VEC ? weight_at<P>(at[i / P * P]) + weight_at<P>(i % P) : at[i]];
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const int a = VEC && IL ? 2 * j : j, e = VEC && IL ? 2 * j + 1 : P + j;
                    const float u = x[a], v = x[e];
                    x[a] = u * cs[j] - v * sn[j];
                    x[e] = v * cs[j] + u * sn[j];
                }
                void *dst = is_q ? p.qo : p.ko;
                const int type = is_q ? p.q_type : p.k_type;
                const int64_t base = is_q ? t * p.qo_st + h * p.qo_sh : t * p.ko_st + (h - p.hq) * p.ko_sh;
                if (VEC) {
                    store_run<P>(dst, base + at[0], type, &x[0]);
                    store_run<P>(dst, base + at[P], type, &x[P]);
                } else {
#pragma unroll
                    for (int j = 0; j < P; ++j)
                        if (p0 + j < half_d) {
                            store1(dst, base + at[j], type, x[j]);
                            store1(dst, base + at[P + j], type, x[P + j]);
                        }
                }
            }
        }
    }
}

int size_of(int type) { return type == CQ_T_F32 ? 4 : 2; }

template <typename T, int P>
void launch_p(const RopeParams &p, bool il, bool vec, int grid, cudaStream_t st) {
    if (il && vec) qk_norm_rope_kernel<T, P, true, true><<<grid, kThreads, 0, st>>>(p);
    else if (vec) qk_norm_rope_kernel<T, P, false, true><<<grid, kThreads, 0, st>>>(p);
    else if (il) qk_norm_rope_kernel<T, 4, true, false><<<grid, kThreads, 0, st>>>(p);
    else qk_norm_rope_kernel<T, 4, false, false><<<grid, kThreads, 0, st>>>(p);
}
template <typename T>
void launch_t(const RopeParams &p, int pairs, bool il, bool vec, int grid, cudaStream_t st) {
    if (sizeof(T) == 2 && pairs == 8) launch_p<T, sizeof(T) == 2 ? 8 : 4>(p, il, vec, grid, st);
    else launch_p<T, 4>(p, il, vec, grid, st);
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
    // Runs of P elements need every offset of a run to be a multiple of P: 8 of a 16-bit type, else 4, else single elements.
    const bool il = d.interleaved != 0;
    auto fits = [&](int P) {
        bool ok = il ? d.head_dim % (2 * P) == 0 : (d.rot_dim / 2) % P == 0 && (d.head_dim - d.rot_dim) / 2 % P == 0;
        auto runs = [&](const void *b, int64_t st, int64_t sh, int type, int heads) {
            const int bytes = std::min(16, P * size_of(type));
            ok = ok && (!heads || (reinterpret_cast<uintptr_t>(b) % bytes == 0 && st * size_of(type) % bytes == 0 && sh * size_of(type) % bytes == 0));
        };
        runs(p.q, p.q_st, p.q_sh, d.in_dtype, d.n_q_heads);
        runs(p.k, p.k_st, p.k_sh, d.in_dtype, d.n_kv_heads);
        runs(p.qo, p.qo_st, p.qo_sh, p.q_type, d.n_q_heads);
        runs(p.ko, p.ko_st, p.ko_sh, p.k_type, d.n_kv_heads);
        return ok;
    };
    const int pairs = d.in_dtype != CQ_T_F32 && fits(8) ? 8 : 4;
    const bool vec = pairs == 8 || fits(4);
    const int lanes = (d.head_dim / 2 + pairs - 1) / pairs;
    p.log_g = 0;
    while ((1 << p.log_g) < lanes) ++p.log_g;
    // A warp takes as many of a token's heads as still leave every SM 32 warps.
    const int slots = 32 >> p.log_g, sms = sm_count();
    p.chunk = slots;
    while (p.chunk < p.heads && (long long)p.tokens * ((p.heads + 2 * p.chunk - 1) / (2 * p.chunk)) >= 32LL * sms) p.chunk *= 2;
    p.chunks = (p.heads + p.chunk - 1) / p.chunk;
    const long long blocks = ((long long)p.tokens * p.chunks + kWarps - 1) / kWarps;
    const int grid = (int)std::min<long long>(blocks, (long long)kBlocks * sms);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (d.in_dtype == CQ_T_F32) launch_t<float>(p, 4, il, vec, grid, st);
    else if (d.in_dtype == CQ_T_F16) launch_t<__half>(p, pairs, il, vec, grid, st);
    else launch_t<__nv_bfloat16>(p, pairs, il, vec, grid, st);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return set_error(CQ_ERR_CUDA, "norm and rotation launch: %s", cudaGetErrorString(e));
    return CQ_OK;
}

}  // namespace cq
