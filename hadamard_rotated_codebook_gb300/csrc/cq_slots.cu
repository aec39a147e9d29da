// cq_slots.cu -- keys and values quantised into the rows of a paged CQ cache.
//
// Per group of 128: r = x H / sqrt(128), n = |x| stored as fp16, and each
// coordinate's code is the number of midpoints m between neighbouring levels
// with r > m * max(n, 1e-12) (a tie falls to the lower level).
//
// Eight lanes own a group, 16 consecutive coordinates each: four stages of the
// transform in registers, three by shuffles, and a warp stores four groups' codes as
// whole words. A code is found by binary search (2 to 4 steps, the midpoints in shared
// memory as a heap: at most 8 different words a step, never two in a bank).
//
// Decisions are those of exact arithmetic. In fp32 the seven stages and the
// scaling are off by at most 8 roundings of 2^-24 of n (every partial sum is at most
// n after scaling), 1/n by 7 and the quotient by 1: 16 in all, under 1e-6. The two
// midpoints next to a coordinate lie on its search path, so the path tells whether it
// is within 1e-6 of one; then, or where n lies within 1e-6 of a border between two fp16
// values, those coordinates and the norm are computed again in fp64. For Gaussian rows that is
// about 1% of the groups, and mostly one coordinate of them, so its sum is taken directly (the
// transform of the whole group in fp64, at this GPU's sixty-fourth of the fp32 rate, would cost as
// much as all the rest).
//
// Bound by instructions (150 a group at four bits, 100 at three), not by memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "cq_paged.h"

namespace cq {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr float kNear = 1e-6f;
constexpr float kInvSqrt128 = 0.08838834764831845f;

struct SideParams {
    uint8_t *codes;
    __half *norms;
    const void *rows;
    int64_t stride;
    int width, groups, bits;
    bool vec;            // rows start on 16-byte boundaries
    long long warps;     // of four groups each
    float heap[16];      // midpoints as a search heap: node 1 the middle one, children of k at 2k and 2k + 1
    double mid[15];
};

struct SlotParams {
    SideParams side[2];
    const int32_t *slots;
    unsigned int *status;
    int cap, n;
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

// 16 consecutive elements, zero past `have`.
template <typename T>
__device__ __forceinline__ void load16(const T *src, int have, bool vec, float (&x)[16]) {
    if (vec && have >= 16) {
        constexpr int kPer = 16 / sizeof(T);
#pragma unroll
        for (int i = 0; i < 16 / kPer; ++i) {
            const uint4 v = reinterpret_cast<const uint4 *>(src)[i];
            const T *e = reinterpret_cast<const T *>(&v);
#pragma unroll
            for (int j = 0; j < kPer; ++j) x[i * kPer + j] = to_f(e[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = j < have ? to_f(src[j]) : 0.0f;
    }
}

// The near coordinates (bits of `near`) and the norm of a warp's groups again, exactly: a coordinate is the sum of its
// group's elements with the signs of the Hadamard matrix, 16 terms a lane, one coordinate of each group at a time.
template <typename T>
__device__ __noinline__ void decide(const SideParams &s, const T *src, int have, int levels, unsigned near, uint64_t &codes, int w, __half &norm) {
    const int lane = threadIdx.x & 31, sub = lane & 7;
    double m2 = 0.0;
#pragma unroll 1
    for (int j = 0; j < 16; ++j) {
        const double x = j < have ? (double)to_f(src[j]) : 0.0;
        m2 = fma(x, x, m2);
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m2 += __shfl_xor_sync(0xFFFFFFFFu, m2, o);
    const double m = sqrt(m2), border = fmax(m, 1e-12) * 11.313708498984761;  // the sums below are unscaled
    norm = __float2half_rn((float)m);  // fp32, then fp16, as the format says
#pragma unroll 1
    while (__any_sync(0xFFFFFFFFu, near)) {
        const unsigned has = __ballot_sync(0xFFFFFFFFu, near) >> (lane & 24) & 0xFFu;  // lanes of this group with one left
        const int owner = has ? __ffs(has) - 1 : 0;
        const int bit = __shfl_sync(0xFFFFFFFFu, __ffs(near) - 1, (lane & 24) + owner) & 15, k = 16 * owner + bit;
        double r = 0.0;
#pragma unroll 1
        for (int j = 0; j < 16; ++j) {
            const double x = j < have ? (double)to_f(src[j]) : 0.0;
            r += __popc(k & (16 * sub + j)) & 1 ? -x : x;
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) r += __shfl_xor_sync(0xFFFFFFFFu, r, o);
        if (has && sub == owner) {
            int c = 0;
            for (int l = 0; l < levels - 1; ++l) c += r > s.mid[l] * border;
            if (levels == 3) c = (c - 1) & 3;
            codes = (codes & ~((uint64_t)((1 << w) - 1) << (bit * w))) | (uint64_t)c << (bit * w);
            near &= near - 1;
        }
    }
}

template <int LEVELS, typename T>
__device__ __forceinline__ void encode(const SlotParams &p, const SideParams &s, const float *heap, long long warp_task, int lane) {
    constexpr int W = LEVELS == 16 ? 4 : LEVELS == 8 ? 3 : 2;
    const int sub = lane & 7;
    const long long task = warp_task * 4 + (lane >> 3);
    int i, g;
    if (s.warps < 1 << 29) {  // the usual case: a 32-bit division
        const unsigned t = (unsigned)task;
        i = (int)min((unsigned)p.n - 1, t / (unsigned)s.groups), g = (int)(t % (unsigned)s.groups);
    } else {
        i = (int)min((long long)p.n - 1, task / s.groups), g = (int)(task % s.groups);
    }
    const int slot = p.slots[i];
    const bool mine = task < (long long)p.n * s.groups, live = mine && slot >= 0 && slot < p.cap;
    if (mine && !live && slot != -1 && sub == 0) atomicOr(p.status, kStatusIndex);
    if (!__any_sync(0xFFFFFFFFu, live)) return;
    const int k0 = g * kGroup + 16 * sub, have = live ? s.width - k0 : 0;
    const T *src = static_cast<const T *>(s.rows) + i * s.stride + k0;
    float x[16], n2 = 0.0f;
    load16(src, have, s.vec, x);
#pragma unroll
    for (int j = 0; j < 16; ++j) n2 = fmaf(x[j], x[j], n2);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) n2 += __shfl_xor_sync(0xFFFFFFFFu, n2, o);
#pragma unroll
    for (int h = 1; h < 16; h <<= 1)
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (!(j & h)) {
                const float a = x[j], b = x[j + h];
                x[j] = a + b, x[j + h] = a - b;
            }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
        const float sign = (sub & o) ? -1.0f : 1.0f;
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = fmaf(x[j], sign, __shfl_xor_sync(0xFFFFFFFFu, x[j], o));
    }
    const float n = sqrtf(n2), scale = kInvSqrt128 / fmaxf(n, 1e-12f);
    unsigned near = 0;
    uint64_t codes = 0;
    const float first = heap[1];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const float u = x[j] * scale;
        int c;
        float dist;
        if (LEVELS == 3) {
            const float a = u - heap[1], b = u - heap[2];
            c = ((a > 0.0f) + (b > 0.0f) - 1) & 3;
            dist = fminf(fabsf(a), fabsf(b));
        } else {
            float d = u - first;
            dist = fabsf(d);
            int k = d > 0.0f ? 3 : 2;
#pragma unroll
            for (int l = 1; l < W; ++l) {
                d = u - heap[k];
                dist = fminf(dist, fabsf(d));
                k = 2 * k + (d > 0.0f);
            }
            c = k - LEVELS;
        }
        near |= (unsigned)(dist <= kNear) << j;
        codes |= (uint64_t)(unsigned)c << (j * W);
    }
    __half norm = __float2half_rn(n);
    bool wild = n2 < 1e-30f || n2 > 1e30f;  // a sum of squares that fp32 may not hold
    if (__any_sync(0xFFFFFFFFu, wild)) {
        // a group of zeros is decided as it stands (every coordinate is exactly zero); else every coordinate again
        bool nonzero = false;
#pragma unroll
        for (int j = 0; j < 16; ++j) nonzero |= x[j] != 0.0f;
        nonzero = __ballot_sync(0xFFFFFFFFu, nonzero) >> (lane & 24) & 0xFFu;
        if (wild) near = nonzero ? 0xFFFFu : 0u;
    }
    const bool edge = __half_as_ushort(__float2half_rn(n * (1.0f + kNear))) != __half_as_ushort(__float2half_rn(n * (1.0f - kNear)));
    if (!live) near = 0;
    if (__any_sync(0xFFFFFFFFu, near || (edge && live))) decide<T>(s, src, have, LEVELS, near, codes, W, norm);
    if (!live) return;
    const size_t at = (size_t)slot * s.groups + g;
    if (sub == 0) s.norms[at] = norm;
    uint8_t *dst = s.codes + at * (16 * W) + sub * 2 * W;
    if (W == 2) {
        *reinterpret_cast<uint32_t *>(dst) = (uint32_t)codes;
    } else if (W == 4) {
        *reinterpret_cast<uint2 *>(dst) = make_uint2((uint32_t)codes, (uint32_t)(codes >> 32));
    } else {
#pragma unroll
        for (int k = 0; k < 3; ++k) reinterpret_cast<uint16_t *>(dst)[k] = (uint16_t)(codes >> (16 * k));
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) kv_write_slots_kernel(const __grid_constant__ SlotParams p) {
    __shared__ float heap[2][16];
    const int tid = threadIdx.x, lane = tid & 31;
    if (tid < 32) heap[tid >> 4][tid & 15] = p.side[tid >> 4].heap[tid & 15];
    __syncthreads();
    const long long all = p.side[0].warps + p.side[1].warps;
    for (long long t = (long long)blockIdx.x * kWarps + (tid >> 5); t < all; t += (long long)gridDim.x * kWarps) {
        const int which = t >= p.side[0].warps;
        const SideParams &s = p.side[which];
        const long long task = which ? t - p.side[0].warps : t;
        switch (s.bits) {
        case 2: encode<4, T>(p, s, heap[which], task, lane); break;
        case 3: encode<8, T>(p, s, heap[which], task, lane); break;
        case 4: encode<16, T>(p, s, heap[which], task, lane); break;
        default: encode<3, T>(p, s, heap[which], task, lane); break;
        }
    }
}

}  // namespace

int launch_kv_write_slots(const SlotSide side[2], int cap, int dtype, const int32_t *slots, int n, void *stream) {
    SlotParams p;
    const int size = dtype == CQ_T_F32 ? 4 : 2;
    for (int i = 0; i < 2; ++i) {
        const SlotSide &a = side[i];
        SideParams &s = p.side[i];
        s.codes = a.codes;
        s.norms = reinterpret_cast<__half *>(a.norms);
        s.rows = a.rows;
        s.stride = a.stride;
        s.width = a.width, s.groups = a.groups, s.bits = a.bits;
        s.vec = reinterpret_cast<uintptr_t>(a.rows) % 16 == 0 && (a.stride * size % 16 == 0 || n == 1);
        s.warps = ((long long)n * a.groups + 3) / 4;
        const int levels = levels_of(a.bits);
        for (int l = 0; l < 16; ++l) s.heap[l] = 0.0f;
        for (int l = 0; l + 1 < levels; ++l) s.mid[l] = 0.5 * ((double)a.codebook[l] + (double)a.codebook[l + 1]);
        if (levels == 3) {
            s.heap[1] = (float)s.mid[0], s.heap[2] = (float)s.mid[1];
        } else {
            for (int step = levels / 2, k = 1; step; step /= 2)  // a level of the heap: every (2 step)-th midpoint from step - 1 on
                for (int l = step - 1; l < levels - 1; l += 2 * step) s.heap[k++] = (float)s.mid[l];
        }
    }
    p.slots = slots;
    p.cap = cap;
    p.n = n;
    p.status = device_status_ptr();
    if (!p.status) return set_error(CQ_ERR_CUDA, "no device status word");
    const long long blocks = (p.side[0].warps + p.side[1].warps + kWarps - 1) / kWarps;
    const int grid = (int)std::min<long long>(blocks, 8LL * sm_count());
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == CQ_T_F32) kv_write_slots_kernel<float><<<grid, kThreads, 0, st>>>(p);
    else if (dtype == CQ_T_F16) kv_write_slots_kernel<__half><<<grid, kThreads, 0, st>>>(p);
    else kv_write_slots_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return set_error(CQ_ERR_CUDA, "slot write launch: %s", cudaGetErrorString(e));
    return CQ_OK;
}

}  // namespace cq
