// cq_norm.cu -- a block's output onto the residual stream, and the next block's norm of the sum.
//
//   z = x / sqrt(mean(x^2) + eps) * (offset + wb)   (or x * (offset + wb), or x)
//   r = residual_scale * res + branch_scale * act(gate) z
//   y = r / sqrt(mean(r^2) + eps) * (offset + w),   or int8 codes of y with a scale per row
//
// A row's second mean needs all of r, so a row stays in registers: a team of lanes (a warp for rows of up to 512
// elements, else a block) owns a row, a lane has CH runs of 8 elements, and every element is read once and written
// once. Teams walk over the rows; the rows to come are on their way into a ring in shared memory by bulk copies (one
// instruction a tensor and row) while the reductions of this one wait on each other. Rows that are not whole 16-byte
// units are read element by element instead. Which lane adds which element depends on the row's width alone, so a
// row's bits depend neither on the other rows nor on how it is aligned.
//
// Codes: y_k = inv * t_k, t_k = r_k (offset + w_k). A product with one positive factor keeps the order of its values, so the
// largest |y| is inv * max|t|, rounded, and the maximum is reduced together with the sum of squares. Scale and codes then
// are those of cq_act_quant_int8 over the fp32 y, bit for bit. A code is the rounded product with the scale's reciprocal, and the rounded
// quotient only where that lies next to a tie (store_codes): a division per element took 88 us where this takes 61.
//
// The bound is memory, and issue slots next to it (two elements to an instruction where there is one for that). 8190 rows of
// 4096 in fp32 onto bf16 with a norm of the branch, to int8 (302 MB): 61 us, 5.0 TB/s or 73% of the copy rate; 16383 of 2048 in bf16 with
// a silu gate for every element (336 MB): 69 us, 72%, issue slots at 68%; 8190 of 4096 in bf16 without either: 47 us, 84%. Steps of a
// few rows take 3 to 5 us, which is two latencies of memory and the launch. Rows of 16384 in fp32 leave the ring one stage
// (129 us for 2048 of them with a norm of the branch, 61%), and 40000 of 333 in fp32, read element by element, take 86 us (36%).
// Tried and slower: four runs a lane instead of two (94 against 69 us: half as many warps wait), one run a lane (78
// against 61 us to int8: an element costs more instructions, though single rows are 0.5 us faster), weights loaded before the reductions (76 us: registers).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "cq_layer.h"

namespace cq {
namespace {

constexpr int kRun = 8;          // consecutive elements of a lane's run
constexpr int kWarpRow = 512;    // widest row that a warp takes alone (777 rows of 1000: 7.4 us with a warp each, 5.2 with two)
constexpr int kWarpTeams = 4;    // such rows of a block
constexpr int kMaxWarps = 16;    // of a block that takes a row
constexpr int kMaxDepth = 4;
constexpr unsigned kSpin = 1u << 20;
constexpr int ring_bytes(int per_sm) { return 228 * 1024 / per_sm - 2048; }  // of a block: a kilobyte is the system's, less than one the barriers'
static_assert(CQ_NORM_MAX_WIDTH <= 32 * kMaxWarps * 4 * kRun, "a block's lanes hold a row");
static_assert(CQ_NORM_MAX_WIDTH * 12 <= ring_bytes(1), "a ring holds a row of each input in fp32");

struct NormParams {
    const void *x, *res, *gate;
    const float *w, *wb;
    void *sum, *y;
    float *scale;
    int64_t x_st, res_st, gate_st, sum_st, y_st;
    int rows, d;
    int x_type, res_type, y_type;
    int act;
    bool post, one_gate;  // one_gate: a gate per row
    float eps, offset, branch, keep, inv_d;
    unsigned int *status;
    unsigned spin;        // polls after which a wait gives up
    bool give_up;         // waits are for what never lands (a self-test)
    int depth;            // stages of a team's ring
    int stage, at_res, at_gate;  // bytes of a stage; where its tensors begin
};

// A run as it comes from memory: 16 bytes of a 16-bit type, 32 of fp32.
struct Raw {
    uint4 a, b;
};
__device__ __forceinline__ float load_one(const void *base, int64_t off, int type) {
    if (type == CQ_T_F32) return static_cast<const float *>(base)[off];
    if (type == CQ_T_F16) return __half2float(static_cast<const __half *>(base)[off]);
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(base)[off]);
}
// A run read element by element: n of its 8 exist.
__device__ __forceinline__ void load_each(Raw &r, const void *base, int64_t off, int type, int n) {
    uint32_t v[kRun];
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
        v[j] = 0;
        if (j < n) v[j] = type == CQ_T_F32 ? static_cast<const uint32_t *>(base)[off + j] : static_cast<const uint16_t *>(base)[off + j];
    }
    if (type == CQ_T_F32) {
        r.a = make_uint4(v[0], v[1], v[2], v[3]), r.b = make_uint4(v[4], v[5], v[6], v[7]);
    } else {
        r.a = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
        r.b = make_uint4(0, 0, 0, 0);
    }
}
// Two fp32 operations in one instruction; a run is four such pairs.
struct F2 {
    uint64_t v;
};
constexpr int kPairs = kRun / 2;
__device__ __forceinline__ F2 f2(float x, float y) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};\n" : "=l"(r.v) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 f2_get(F2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;\n" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 f2_add(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ void unpack(const Raw &r, int type, F2 (&v)[kPairs]) {
    const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
    if (type == CQ_T_F32) {
#pragma unroll
        for (int j = 0; j < kPairs; ++j) v[j] = f2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
    } else if (type == CQ_T_F16) {
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[j]));
            v[j] = f2(f.x, f.y);
        }
    } else {
#pragma unroll
        for (int j = 0; j < kPairs; ++j) v[j] = f2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
    }
}
template <bool VEC>
__device__ __forceinline__ void store_run(void *base, int64_t off, int type, const F2 (&v)[kPairs], int n) {
    uint32_t w[kRun];
    if (type == CQ_T_F32) {
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            const float2 f = f2_get(v[j]);
            w[2 * j] = __float_as_uint(f.x), w[2 * j + 1] = __float_as_uint(f.y);
        }
    } else {
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            const float2 f = f2_get(v[j]);
            if (type == CQ_T_F16) {
                const __half2 h = __floats2half2_rn(f.x, f.y);
                w[j] = *reinterpret_cast<const uint32_t *>(&h);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
                w[j] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
    }
    if (VEC) {
        uint4 *p = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(base) + off * (type == CQ_T_F32 ? 4 : 2));
        p[0] = make_uint4(w[0], w[1], w[2], w[3]);
        if (type == CQ_T_F32) p[1] = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
#pragma unroll
        for (int j = 0; j < kRun; ++j) {
            if (j >= n) continue;
            if (type == CQ_T_F32) static_cast<uint32_t *>(base)[off + j] = w[j];
            else static_cast<uint16_t *>(base)[off + j] = (uint16_t)(w[j / 2] >> (16 * (j & 1)));
        }
    }
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// rint(v / step), v / step rounded to fp32 first, as bytes. Where the product with step's reciprocal is further than
// kNear from a tie it decides: it and the rounded quotient are off by 2^-23 and 2^-24 of at most 127.5, 2.3e-5 together.
// Adding 1.5 * 2^23 leaves the nearest integer in the low bits. `plain`: the row's quotients are at most 127.5 and
// the reciprocal a normal number.
constexpr float kNear = 4e-5f, kMagic = 12582912.0f;
template <bool VEC>
__device__ __forceinline__ void store_codes(int8_t *dst, const F2 (&v)[kPairs], float step, float back, bool plain, int n) {
    uint32_t q[kRun];
    float far = 0.0f;
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
        const F2 t = f2_mul(v[j], f2(back, back)), m = f2_add(t, f2(kMagic, kMagic));
        const float2 d = f2_get(f2_fma(f2_add(m, f2(-kMagic, -kMagic)), f2(-1.0f, -1.0f), t)), i = f2_get(m);
        far = max_nan(far, max_nan(fabsf(d.x), fabsf(d.y)));
        q[2 * j] = __float_as_uint(i.x), q[2 * j + 1] = __float_as_uint(i.y);
    }
    if (!plain || !(far <= 0.5f - kNear)) {  // no number counts as near
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            const float2 f = f2_get(v[j]);
            q[2 * j] = (uint32_t)(int)fminf(fmaxf(rintf(__fdiv_rn(f.x, step)), -128.0f), 127.0f);
            q[2 * j + 1] = (uint32_t)(int)fminf(fmaxf(rintf(__fdiv_rn(f.y, step)), -128.0f), 127.0f);
        }
    }
    uint32_t w[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
        w[j] = __byte_perm(__byte_perm(q[4 * j], q[4 * j + 1], 0x0040), __byte_perm(q[4 * j + 2], q[4 * j + 3], 0x0040), 0x5410);
    if (VEC) {
        *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int j = 0; j < kRun; ++j)
            if (j < n) dst[j] = (int8_t)(w[j / 4] >> (8 * (j & 3)));
    }
}
// offset + weight (zero past the row).
template <bool VEC>
__device__ __forceinline__ void load_weight(const float *w, int n, float offset, F2 (&t)[kPairs]) {
    if (VEC) {
        const float4 a = __ldg(reinterpret_cast<const float4 *>(w)), b = __ldg(reinterpret_cast<const float4 *>(w) + 1);
        t[0] = f2(a.x, a.y), t[1] = f2(a.z, a.w), t[2] = f2(b.x, b.y), t[3] = f2(b.z, b.w);
    } else {
#pragma unroll
        for (int j = 0; j < kPairs; ++j) t[j] = f2(2 * j < n ? __ldg(w + 2 * j) : 0.0f, 2 * j + 1 < n ? __ldg(w + 2 * j + 1) : 0.0f);
    }
    if (offset != 0.0f) {
#pragma unroll
        for (int j = 0; j < kPairs; ++j) t[j] = f2_add(t[j], f2(offset, offset));
    }
}

// 1 / (1 + 2^(-g log2 e)); beyond the range of the power it is 0 or 1.
__device__ __forceinline__ float sigmoid(float g) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(e) : "f"(g * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(1.0f + e));
    return r;
}
__device__ __forceinline__ float open(float g, int act) {
    return act == CQ_GATE_PLAIN ? g : act == CQ_GATE_SIGMOID ? sigmoid(g) : g * sigmoid(g);
}

__device__ __forceinline__ float warp_max(float x) {  // of values that are not below zero: ordered as integers; NaNs are not among them
    return __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(x)));
}
// Sum of s and maximum of m (not below zero) over the team. Block teams: one barrier, the warps' parts in a buffer that alternates.
template <bool WARP>
__device__ __forceinline__ void reduce(float &s, float &m, bool with_max, float2 *buf) {
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (with_max) m = warp_max(m);
    if (WARP) return;
    const int warps = blockDim.x >> 5, all = 1 << (32 - __clz(warps - 1)), part = threadIdx.x & (all - 1);  // (a block has two warps and more)
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = make_float2(s, m);
    __syncthreads();
    const float2 v = part < warps ? buf[part] : make_float2(0.0f, 0.0f);  // every `all` lanes hold them all
    s = v.x;
#pragma unroll 1
    for (int o = all >> 1; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (with_max) m = warp_max(v.y);
}

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void bulk(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(dst), "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
// Starts the copies of a row into a stage of the ring (one lane).
__device__ __forceinline__ void fetch_row(const NormParams &p, int64_t row, uint32_t to, uint32_t bar) {
    const uint32_t nx = p.d * (p.x_type == CQ_T_F32 ? 4 : 2), nr = p.res ? p.d * (p.res_type == CQ_T_F32 ? 4 : 2) : 0;
    const uint32_t ng = p.gate && !p.one_gate ? nx : 0;
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(bar), "r"(nx + nr + ng) : "memory");
    const int64_t size = p.x_type == CQ_T_F32 ? 4 : 2, rsize = p.res_type == CQ_T_F32 ? 4 : 2;
    bulk(to, static_cast<const uint8_t *>(p.x) + row * p.x_st * size, nx, bar);
    if (nr) bulk(to + p.at_res, static_cast<const uint8_t *>(p.res) + row * p.res_st * rsize, nr, bar);
    if (ng) bulk(to + p.at_gate, static_cast<const uint8_t *>(p.gate) + row * p.gate_st * size, ng, bar);
}
__device__ __forceinline__ bool poll(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity), "r"(1000u)
                 : "memory");
    return ok;
}
// A copy that does not land within p.spin polls marks the status word; no wait of the block waits any longer then (false: it has not landed).
__device__ __forceinline__ bool wait(const NormParams &p, uint32_t bar, uint32_t parity, volatile int &abort) {
    for (unsigned i = 0; !poll(bar, parity); ++i) {
        if (abort) return false;
        if (i >= p.spin) {
            atomicOr(p.status, 0x474A0001u);
            abort = 1;
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ void take_run(Raw &r, uint32_t from, int type) {
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n" : "=r"(r.a.x), "=r"(r.a.y), "=r"(r.a.z), "=r"(r.a.w) : "r"(from) : "memory");
    if (type == CQ_T_F32)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n" : "=r"(r.b.x), "=r"(r.b.y), "=r"(r.b.z), "=r"(r.b.w) : "r"(from + 16) : "memory");
}

// Waits (bounded) for copies of a team that gave up, whose ends no wait has seen: those of `row` (none past the last), in stage st with parity par, and of
// the rows after it.
__noinline__ __device__ void land(const NormParams &p, int64_t row, int st, uint32_t par, int64_t teams, uint32_t full) {
    for (int i = 0; i < p.depth && row + i * teams < p.rows; ++i) {
        const int at = st + i;
        for (unsigned k = 0; k < kSpin && !poll(full + 8 * (at % p.depth), par ^ (at >= p.depth)); ++k) {}
    }
}

// VEC: rows are whole runs on 16-byte boundaries and come through the ring. Without a least number of blocks given the compiler takes 2 to 18
// registers fewer, at a price in instructions: 16383 rows of 2048, gated, 71 us against 68, 65536 of 512 54 against 51. Rows read element by
// element want the warps instead (40000 of 333: 95 us with one block, 86 with six).
template <int CH, bool WARP, bool VEC, bool GATE>
__global__ void __launch_bounds__(WARP ? 32 * kWarpTeams : 32 * kMaxWarps, WARP && !VEC ? 6 : 1) block_norm_kernel(const __grid_constant__ NormParams p) {
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float2 s_buf[4][kMaxWarps];
    __shared__ uint64_t s_full[WARP ? kWarpTeams : 1][kMaxDepth];
    __shared__ uint64_t s_never;
    __shared__ volatile int s_left, s_stage;  // of a block that gave up: see land
    __shared__ volatile uint32_t s_par;
    __shared__ volatile int s_abort;
    const int lanes = WARP ? 32 : blockDim.x, lane = WARP ? threadIdx.x & 31 : threadIdx.x, team = WARP ? threadIdx.x >> 5 : 0;
    const int64_t teams = WARP ? gridDim.x * kWarpTeams : gridDim.x;
    int64_t row = WARP ? blockIdx.x * kWarpTeams + team : blockIdx.x;
    const uint32_t mine = smem_u32(ring) + team * p.depth * p.stage, full = smem_u32(s_full[team]);
    if (VEC) {
        if (threadIdx.x == 0) {
            s_abort = 0, s_left = -1;
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;\n" ::"r"(smem_u32(&s_never)));
        }
        if (lane == 0) {
            for (int i = 0; i < p.depth; ++i) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;\n" ::"r"(full + 8 * i));
            asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
            for (int i = 0; i < p.depth && row + i * teams < p.rows; ++i) fetch_row(p, row + i * teams, mine + i * p.stage, full + 8 * i);
        }
        __syncthreads();
    }
    int st = 0;
    uint32_t par = 0;
#pragma unroll 1
    for (int turn = 0; row < p.rows; row += teams, turn ^= 2) {
        const uint32_t from = mine + st * p.stage;
        if (VEC) {
            const bool there = wait(p, p.give_up ? smem_u32(&s_never) : full + 8 * st, par, s_abort);
            if (WARP && !__all_sync(0xFFFFFFFFu, there)) break;  // (a block's teams go on, for their barriers)
        }
        F2 v[CH][kPairs], sum = {0};
        float none = 0.0f, ib = p.branch;  // what a branch's element is multiplied by, but for its weight
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int e = (c * lanes + lane) * kRun, n = p.d - e;
            Raw r = {};
            if (!VEC) load_each(r, p.x, row * p.x_st + e, p.x_type, n);
            else if (n > 0) take_run(r, from + e * (p.x_type == CQ_T_F32 ? 4 : 2), p.x_type);
            unpack(r, p.x_type, v[c]);
        }
        if (p.post) {
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int j = 0; j < kPairs; ++j) sum = f2_fma(v[c][j], v[c][j], sum);
            const float2 two = f2_get(sum);
            float s = two.x + two.y;
            reduce<WARP>(s, none, false, s_buf[turn]);
            ib = rsqrtf(fmaf(s, p.inv_d, p.eps)) * p.branch;
            if (!p.wb) ib *= p.offset + 1.0f;
        }
        if (GATE && p.one_gate) ib *= open(load_one(p.gate, row * p.gate_st, p.x_type), p.act);
        float top = 0.0f;
        sum = f2(0.0f, 0.0f);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int e = (c * lanes + lane) * kRun, n = p.d - e;
            if (n <= 0) continue;
            Raw r = {};
            F2 t[kPairs];
#pragma unroll
            for (int j = 0; j < kPairs; ++j) v[c][j] = f2_mul(v[c][j], f2(ib, ib));
            if (p.wb) {
                load_weight<VEC>(p.wb + e, n, p.offset, t);
#pragma unroll
                for (int j = 0; j < kPairs; ++j) v[c][j] = f2_mul(v[c][j], t[j]);
            }
            if (GATE && !p.one_gate) {
                if (VEC) take_run(r, from + p.at_gate + e * (p.x_type == CQ_T_F32 ? 4 : 2), p.x_type);
                else load_each(r, p.gate, row * p.gate_st + e, p.x_type, n);
                unpack(r, p.x_type, t);
#pragma unroll
                for (int j = 0; j < kPairs; ++j) {
                    const float2 g = f2_get(t[j]);
                    v[c][j] = f2_mul(v[c][j], f2(open(g.x, p.act), open(g.y, p.act)));
                }
            }
            if (p.res) {
                if (VEC) take_run(r, from + p.at_res + e * (p.res_type == CQ_T_F32 ? 4 : 2), p.res_type);
                else load_each(r, p.res, row * p.res_st + e, p.res_type, n);
                unpack(r, p.res_type, t);
#pragma unroll
                for (int j = 0; j < kPairs; ++j) v[c][j] = f2_fma(f2(p.keep, p.keep), t[j], v[c][j]);
            }
            if (!VEC) {  // what is not there may have become no number (0 times an infinity)
#pragma unroll
                for (int j = 0; j < kPairs; ++j) {
                    const float2 f = f2_get(v[c][j]);
                    v[c][j] = f2(2 * j < n ? f.x : 0.0f, 2 * j + 1 < n ? f.y : 0.0f);
                }
            }
            if (p.sum) store_run<VEC>(p.sum, row * p.sum_st + e, p.res_type, v[c], n);
            if (p.w) {
                load_weight<VEC>(p.w + e, n, p.offset, t);
            } else {
#pragma unroll
                for (int j = 0; j < kPairs; ++j) t[j] = f2(p.offset + 1.0f, p.offset + 1.0f);
            }
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                sum = f2_fma(v[c][j], v[c][j], sum);
                v[c][j] = f2_mul(v[c][j], t[j]);
            }
            if (p.scale) {
#pragma unroll
                for (int j = 0; j < kPairs; ++j) {
                    const float2 f = f2_get(v[c][j]);
                    top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                }
            }
        }
        const float2 two = f2_get(sum);
        float s = two.x + two.y;
        reduce<WARP>(s, top, p.scale != nullptr, s_buf[turn + 1]);  // every lane has read its part of the stage
        if (VEC) {
            const int64_t ahead = row + p.depth * teams;
            if (lane == 0) {
                if (WARP || !s_abort) {
                    if (ahead < p.rows) fetch_row(p, ahead, from, full + 8 * st);
                } else if (s_left < 0) {
                    s_left = (int)row, s_stage = st, s_par = par;
                }
            }
            if (++st == p.depth) st = 0, par ^= 1;
        }
        const float inv = rsqrtf(fmaf(s, p.inv_d, p.eps));
        const float most = top * inv, step = most > 0.0f ? __fdiv_rn(most, 127.0f) : 1.0f, back = 1.0f / step;
        const bool plain = step > 1e-36f && step < 1e36f;
        if (p.scale && lane == 0) p.scale[row] = step;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int e = (c * lanes + lane) * kRun, n = p.d - e;
            if (n <= 0) continue;
#pragma unroll
            for (int j = 0; j < kPairs; ++j) v[c][j] = f2_mul(v[c][j], f2(inv, inv));
            if (p.scale) store_codes<VEC>(static_cast<int8_t *>(p.y) + row * p.y_st + e, v[c], step, back, plain, n);
            else store_run<VEC>(p.y, row * p.y_st + e, p.y_type, v[c], n);
        }
    }
    if (VEC && WARP && lane == 0) land(p, row, st, par, teams, full);
    if (VEC && !WARP && lane == 0 && s_abort && s_left >= 0) land(p, s_left, s_stage, s_par, teams, full);
}

template <int CH, bool WARP, bool VEC, bool GATE>
int launch_k(const NormParams &p, int grid, int threads, cudaStream_t st) {
    const size_t smem = VEC ? (size_t)p.stage * p.depth * (WARP ? kWarpTeams : 1) : 0;
    auto k = block_norm_kernel<CH, WARP, VEC, GATE>;
    if (smem > 32 * 1024) {
        const int rc = ensure_smem(reinterpret_cast<const void *>(k), ring_bytes(1));
        if (rc) return rc;
    }
    k<<<grid, threads, smem, st>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return set_error(CQ_ERR_CUDA, "block norm launch: %s", cudaGetErrorString(e));
    return CQ_OK;
}
template <int CH, bool WARP>
int launch_c(const NormParams &p, bool vec, int grid, int threads, cudaStream_t st) {
    if (vec) return p.gate ? launch_k<CH, WARP, true, true>(p, grid, threads, st) : launch_k<CH, WARP, true, false>(p, grid, threads, st);
    return p.gate ? launch_k<CH, WARP, false, true>(p, grid, threads, st) : launch_k<CH, WARP, false, false>(p, grid, threads, st);
}

int size_of(int type) { return type == CQ_T_F32 ? 4 : type == CQ_T_I8 ? 1 : 2; }

}  // namespace

int launch_block_norm(const cq_norm_desc &d, bool give_up, void *stream) {
    NormParams p;
    p.x = d.x, p.res = d.residual, p.gate = d.gate, p.w = d.weight, p.wb = d.branch_weight;
    p.sum = d.residual_out, p.y = d.out, p.scale = d.out_dtype == CQ_T_I8 ? d.out_scale : nullptr;
    p.x_st = d.x_stride, p.res_st = d.residual_stride, p.gate_st = d.gate_stride, p.sum_st = d.residual_out_stride, p.y_st = d.out_stride;
    p.rows = d.n_tokens, p.d = d.width;
    p.x_type = d.x_dtype, p.res_type = d.residual_dtype, p.y_type = d.out_dtype;
    p.act = d.gate_act, p.post = d.post_norm != 0, p.one_gate = d.gate && d.gate_width == 1;
    p.eps = d.eps, p.offset = d.weight_offset, p.branch = d.branch_scale, p.keep = d.residual_scale;
    p.inv_d = 1.0f / (float)d.width;
    p.status = device_status_ptr();
    p.spin = give_up ? 4 : kSpin, p.give_up = give_up;
    if (!p.status) return set_error(CQ_ERR_CUDA, "no device status word");
    // Rows in bulk copies and 16-byte accesses (8 of int8) need every row to start on such a boundary.
    bool vec = d.width % kRun == 0;
    auto runs = [&](const void *b, int64_t st, int type) {
        const int bytes = std::min(16, kRun * size_of(type));
        vec = vec && (!b || (reinterpret_cast<uintptr_t>(b) % bytes == 0 && (d.n_tokens == 1 || st * size_of(type) % bytes == 0)));
    };
    runs(p.x, p.x_st, p.x_type);
    runs(p.res, p.res_st, p.res_type);
    if (!p.one_gate) runs(p.gate, p.gate_st, p.x_type);
    runs(p.sum, p.sum_st, p.res_type);
    runs(p.y, p.y_st, p.y_type);
    runs(p.w, 0, CQ_T_F32);
    runs(p.wb, 0, CQ_T_F32);
    const int chunks = (d.width + kRun - 1) / kRun, sms = sm_count();
    p.at_res = p.d * size_of(p.x_type);
    p.at_gate = p.at_res + (p.res ? p.d * size_of(p.res_type) : 0);
    p.stage = p.at_gate + (p.gate && !p.one_gate ? p.d * size_of(p.x_type) : 0);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (d.width <= kWarpRow) {
        const int per_sm = 12;  // 65536 rows of 512 in bf16: 51 us; 54 with 10, 55 with 24
        p.depth = std::max(1, std::min(kMaxDepth, ring_bytes(per_sm) / kWarpTeams / p.stage));
        const int grid = (int)std::min<long long>(((long long)p.rows + kWarpTeams - 1) / kWarpTeams, (long long)sms * per_sm);
        return chunks <= 32 ? launch_c<1, true>(p, vec, grid, 32 * kWarpTeams, st) : launch_c<2, true>(p, vec, grid, 32 * kWarpTeams, st);
    }
    const int ch = chunks <= 2 * 32 * kMaxWarps ? 2 : 4, threads = ((chunks + ch - 1) / ch + 31) / 32 * 32;
    // Blocks of an SM before stages of a block: the prompt of 8190 rows of 4096 takes 61 us with four blocks of two stages, 69 with three of
    // three, 81 with two of four (the reductions of more rows overlap).
    int per_sm = std::max(1, std::min(16, 1024 / threads));
    while (per_sm > 1 && ring_bytes(per_sm) / p.stage < 2) --per_sm;
    p.depth = std::max(1, std::min(kMaxDepth, ring_bytes(per_sm) / p.stage));
    const int grid = std::min(p.rows, per_sm * sms);
    return ch == 2 ? launch_c<2, false>(p, vec, grid, threads, st) : launch_c<4, false>(p, vec, grid, threads, st);
}

}  // namespace cq
