// cq_slots.cu -- keys and values quantised into the rows of a paged CQ cache.
//
// Per group of 128: r = x H / sqrt(128), n = |x| stored as fp16, and each
// coordinate's code is the number of midpoints m between neighbouring levels
// with r > m * max(n, 1e-12) (a tie falls to the lower level). A warp owns a
// group, four coordinates a lane: two stages of the transform in registers, five
// by shuffles.
//
// Decisions are those of exact arithmetic. In fp32 the seven stages and the
// scaling are off by at most 8 roundings of 2^-24 of n (every partial sum is at most
// n after scaling), n itself by 5 (times |m| <= 1), m and the difference by 2:
// 15 in all, under 1e-6. Where a coordinate lies within 1e-6 n of a border, or n within
// 1e-6 of a border between two fp16 values, the warp repeats the group in 64 bits. For Gaussian rows that is
// under 1% of the groups.
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

struct SideParams {
    uint8_t *codes;
    __half *norms;
    const void *rows;
    int64_t stride;
    int width, groups, bits;
    bool vec;
    float mid[15];
    double mid64[15];
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

__device__ __forceinline__ void load4(const float *p, float *x) {
    const float4 v = *reinterpret_cast<const float4 *>(p);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
}
template <typename T>
__device__ __forceinline__ void load4(const T *p, float *x) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    const T *h = reinterpret_cast<const T *>(&v);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = to_f(h[j]);
}

// 128-point Sylvester transform over a warp, coordinates 4 * lane + j, unscaled.
template <typename F>
__device__ __forceinline__ void fwht(F (&x)[4], int lane) {
    F a = x[0] + x[1], b = x[0] - x[1], c = x[2] + x[3], d = x[2] - x[3];
    x[0] = a + c, x[1] = b + d, x[2] = a - c, x[3] = b - d;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const F y = __shfl_xor_sync(0xFFFFFFFFu, x[j], o);
            x[j] = (lane & o) ? y - x[j] : x[j] + y;
        }
    }
}

template <int LEVELS, typename T>
__device__ __forceinline__ void encode_group(const SideParams &s, const T *src, int have, int64_t row, int g, int lane) {
    float x[4];
    if (s.vec && have >= 4) {
        load4(src, x);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = j < have ? to_f(src[j]) : 0.0f;
    }
    const float x0[4] = {x[0], x[1], x[2], x[3]};
    float n2 = fmaf(x[0], x[0], x[1] * x[1]) + fmaf(x[2], x[2], x[3] * x[3]);
#pragma unroll
    for (int o = 16; o; o >>= 1) n2 += __shfl_xor_sync(0xFFFFFFFFu, n2, o);
    float n = sqrtf(n2);
    fwht(x, lane);
    constexpr float kInv = 0.08838834764831845f;  // 1/sqrt(128)
    const float nc = fmaxf(n, 1e-12f), eps = kNear * nc;
    int code[4];
    bool near = n2 < 1e-30f || n2 > 1e30f;  // a sum of squares that fp32 may not hold
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float r = x[j] * kInv;
        code[j] = 0;
#pragma unroll
        for (int l = 0; l < LEVELS - 1; ++l) {
            const float d = fmaf(-s.mid[l], nc, r);
            code[j] += d > 0.0f;
            near |= fabsf(d) <= eps;
        }
    }
    __half nh = __float2half_rn(n);
    near |= __half_as_ushort(__float2half_rn(n * (1.0f + kNear))) != __half_as_ushort(__float2half_rn(n * (1.0f - kNear)));
    if (__any_sync(0xFFFFFFFFu, near)) {
        double y[4] = {x0[0], x0[1], x0[2], x0[3]};
        double m2 = y[0] * y[0] + y[1] * y[1] + (y[2] * y[2] + y[3] * y[3]);
#pragma unroll
        for (int o = 16; o; o >>= 1) m2 += __shfl_xor_sync(0xFFFFFFFFu, m2, o);
        const double m = sqrt(m2);
        fwht(y, lane);
        const double border = fmax(m, 1e-12) * 11.313708498984761;  // sqrt(128): the transform above is unscaled
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            code[j] = 0;
#pragma unroll
            for (int l = 0; l < LEVELS - 1; ++l) code[j] += y[j] > s.mid64[l] * border;
        }
        nh = __float2half_rn((float)m);  // fp32, then fp16, as the format says
    }
    if (lane == 0) s.norms[row * s.groups + g] = nh;
    if (LEVELS == 3) {
#pragma unroll
        for (int j = 0; j < 4; ++j) code[j] = (code[j] - 1) & 3;
    }
    constexpr int W = LEVELS == 16 ? 4 : LEVELS == 8 ? 3 : 2;
    const unsigned v = code[0] | code[1] << W | code[2] << 2 * W | code[3] << 3 * W;
    uint8_t *dst = s.codes + (row * s.groups + g) * (16 * W);
    if (W == 2) {
        dst[lane] = (uint8_t)v;
    } else if (W == 4) {
        reinterpret_cast<uint16_t *>(dst)[lane] = (uint16_t)v;
    } else {
        const unsigned w = v | __shfl_down_sync(0xFFFFFFFFu, v, 1) << 12;
        if (!(lane & 1)) {
            dst += 3 * (lane >> 1);
            dst[0] = (uint8_t)w, dst[1] = (uint8_t)(w >> 8), dst[2] = (uint8_t)(w >> 16);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) kv_write_slots_kernel(const __grid_constant__ SlotParams p) {
    const int lane = threadIdx.x & 31;
    const int per = p.side[0].groups + p.side[1].groups;
    const long long tasks = (long long)p.n * per;
    for (long long task = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); task < tasks; task += (long long)gridDim.x * kWarps) {
        const int i = (int)(task / per);
        int g = (int)(task - (long long)i * per);
        const int slot = p.slots[i];
        if (slot < 0 || slot >= p.cap) {
            if (slot != -1 && lane == 0) atomicOr(p.status, kStatusIndex);
            continue;
        }
        const int which = g >= p.side[0].groups;
        const SideParams &s = p.side[which];
        g -= which ? p.side[0].groups : 0;
        const int k0 = g * kGroup + 4 * lane;
        const T *src = static_cast<const T *>(s.rows) + i * s.stride + k0;
        const int have = s.width - k0;
        switch (s.bits) {
        case 2: encode_group<4, T>(s, src, have, slot, g, lane); break;
        case 3: encode_group<8, T>(s, src, have, slot, g, lane); break;
        case 4: encode_group<16, T>(s, src, have, slot, g, lane); break;
        default: encode_group<3, T>(s, src, have, slot, g, lane); break;
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
        s.vec = reinterpret_cast<uintptr_t>(a.rows) % (4 * size) == 0 && (a.stride % 4 == 0 || n == 1);
        for (int l = 0; l + 1 < levels_of(a.bits); ++l) {
            s.mid64[l] = 0.5 * ((double)a.codebook[l] + (double)a.codebook[l + 1]);
            s.mid[l] = (float)s.mid64[l];
        }
    }
    p.slots = slots;
    p.cap = cap;
    p.n = n;
    p.status = device_status_ptr();
    if (!p.status) return set_error(CQ_ERR_CUDA, "no device status word");
    const long long blocks = ((long long)n * (side[0].groups + side[1].groups) + kWarps - 1) / kWarps;
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
