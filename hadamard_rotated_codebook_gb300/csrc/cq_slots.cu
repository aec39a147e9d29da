// cq_slots.cu -- keys and values quantised into the rows of a paged CQ cache.
//
// Per group of 128: r = x H / sqrt(128), n = |x| stored as fp16, and each
// coordinate's code is the number of midpoints m between neighbouring levels
// with r > m * max(n, 1e-12) (a tie falls to the lower level).
//
// Eight lanes own a group, 16 consecutive coordinates each: four stages of the
// transform in registers (two coordinates to an instruction), three by shuffles, and a warp
// stores four groups' codes as whole words. A code is looked up: [-1, 1] is cut into 128
// cells of equal width with at most one midpoint each, and a cell holds that midpoint (or the
// nearest) and the code below it, so that one comparison decides. The table is repeated 16
// times in shared memory, so that no two lanes of half a warp meet in a bank. Codebooks whose
// midpoints lie too close for that are searched instead, over the midpoints as a heap.
//
// Decisions are those of exact arithmetic. In fp32 the seven stages are off by at most 7 roundings
// of 2^-24 of n (every partial sum is at most n after scaling), n by 7 of its own (12 of the sum of
// squares, halved by the root, and the root's), and 1/sqrt(128), the quotient, the product and a
// midpoint by one each: a coordinate next to midpoint m by 2^-24 (7 + 11 |m|) in all, the codebook's
// margin (`near`: 4.6e-7 to 5.7e-7 for the analytic ones, 1.1e-6 for midpoints near 1). No midpoint
// lies within 1/64 of a cell of its edge, so the cell's own midpoint (or the two next to a
// coordinate on its search path) tells whether it is within the margin of one; then, or where n lies
// within 1e-6 of a border between two fp16 values, those coordinates and the norm are computed
// again in fp64. For Gaussian rows that is about 1% of the groups, and mostly one coordinate of
// them, so its sum is taken directly (the transform of the whole group in fp64, at this GPU's
// sixty-fourth of the fp32 rate, would cost as much as all the rest).
//
// Bound by instructions, not by memory: 8190 rows of 8 heads of 128 in bf16, four and three bits (41.2 MB), take 35 us,
// 1.18 TB/s or 17% of the copy rate. 650 instructions go to four groups; issue slots are used to 69%, with 27 warps on an SM
// (58 registers, 33 KB of tables a block), and the fp64 pipe of the exact decisions to 15% of the time (25% at a margin of 1.1e-6
// for every codebook: 36.7 us). A warp that
// decides exactly takes half as long again as the others: dealing a block's tasks out as its warps come for them brought 45.7
// to 35.6 us (before, SMs were busy 54000 to 86000 cycles). A step of 77 rows takes 12 to 13 us, most of it
// setting the tables up and one pass through the code.
// Slower or no faster: a warp to a group (92 us), a binary search for each code (47 against 42 then), loading a task ahead (42),
// 3, 5 or 6 blocks per SM (43 to 49).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "cq_paged.h"

namespace cq {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr float kNear = 1e-6f;           // of a norm: 8 roundings with that of the product
constexpr int kCells = 132;              // 64 to a unit, over [-1, 1] and a margin
constexpr int kCopies = 16;
constexpr int kTable = kCells * kCopies;  // entries of 8 bytes
constexpr float kInvSqrt128 = 0.08838834764831845f;

struct SideParams {
    uint8_t *codes;
    __half *norms;
    const void *rows;
    int64_t stride;
    int width, groups, bits;
    bool vec;            // rows start on 16-byte boundaries
    long long warps;     // of four groups each
    bool cells;          // the cell table holds this codebook
    float heap[16];      // midpoints as a search heap: node 1 the middle one, children of k at 2k and 2k + 1
    float near;          // how far fp32 may be from a coordinate next to a midpoint
    float offset;        // cell of u: the integer part of 64 u + offset - 2^16
    float cell_mid[kCells];
    uint8_t cell_code[kCells];
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

// Two fp32 operations in one instruction.
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 f2(float x, float y) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};\n" : "=l"(r.v) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void f2_get(F2 a, float &x, float &y) { asm("mov.b64 {%0, %1}, %2;\n" : "=f"(x), "=f"(y) : "l"(a.v)); }
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
#pragma unroll 4
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
#pragma unroll 4
        for (int j = 0; j < 16; ++j) {
            const double x = j < have ? (double)to_f(src[j]) : 0.0;
            r += __popc(k & (16 * sub + j)) & 1 ? -x : x;
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) r += __shfl_xor_sync(0xFFFFFFFFu, r, o);
        if (has && sub == owner) {
            // midpoints more than 1e-5 below are counted in fp32, and the few that are left in fp64 (midpoints ascend)
            const float u = border < 1e37 ? (float)r / (float)border : -INFINITY;  // past fp32 all are counted in fp64
            int c = 0;
            for (int l = 0; l < levels - 1; ++l) c += (float)s.mid[l] < u - 1e-5f;
            while (c < levels - 1 && r > s.mid[c] * border) ++c;
            if (levels == 3) c = (c - 1) & 3;
            codes = (codes & ~((uint64_t)((1 << w) - 1) << (bit * w))) | (uint64_t)c << (bit * w);
            near &= near - 1;
        }
    }
}

template <int LEVELS, typename T>
__device__ __forceinline__ void encode(const SlotParams &p, const SideParams &s, const float2 *table, long long warp_task, int lane) {
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
    float x[16];
    load16(src, have, s.vec, x);
    F2 z[8], q2 = f2(0.0f, 0.0f);  // elements 2 j and 2 j + 1
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const F2 v = f2(x[2 * j], x[2 * j + 1]);
        q2 = f2_fma(v, v, q2);
        z[j] = f2(x[2 * j] + x[2 * j + 1], x[2 * j] - x[2 * j + 1]);
    }
    float n2, other;
    f2_get(q2, n2, other);
    n2 += other;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) n2 += __shfl_xor_sync(0xFFFFFFFFu, n2, o);
    const F2 minus = f2(-1.0f, -1.0f);
#pragma unroll
    for (int h = 1; h < 8; h <<= 1)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (!(j & h)) {
                const F2 a = z[j], b = z[j + h];
                z[j] = f2_add(a, b), z[j + h] = f2_fma(b, minus, a);
            }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
        const float sign = (sub & o) ? -1.0f : 1.0f;
        const F2 s2 = f2(sign, sign);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float a, b;
            f2_get(z[j], a, b);
            z[j] = f2_fma(z[j], s2, f2(__shfl_xor_sync(0xFFFFFFFFu, a, o), __shfl_xor_sync(0xFFFFFFFFu, b, o)));
        }
    }
    const float n = sqrtf(n2), scale = kInvSqrt128 / fmaxf(n, 1e-12f);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        f2_get(f2_mul(z[j], f2(scale, scale)), x[2 * j], x[2 * j + 1]);
    }
    unsigned near = 0;
    uint32_t word[2] = {0, 0};  // codes: 16 W bits, the second half from bit 8 W on
    if (s.cells) {
        // 64 u + offset behind 2^16: the sum has seven bits of fraction, so its bits 7 to 14 are the cell, and masked in place
        // the byte offset of the cell's 16 entries of 8 bytes. What is not a number ends in the last cell.
        const char *mine = reinterpret_cast<const char *>(table) + (lane & (kCopies - 1)) * 8;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const float at = fminf(fmaf(x[j], 64.0f, s.offset), 65536.0f + (kCells - 1));
            const float2 e = *reinterpret_cast<const float2 *>(mine + (__float_as_uint(at) & 0x7F80u));
            const float d = x[j] - e.x;
            unsigned c = __float_as_uint(e.y) + (d > 0.0f);
            if (LEVELS == 3) c = (c - 1) & 3;
            word[j / 8] |= c << (j % 8 * W);
            near |= (unsigned)(fabsf(d) <= s.near) << j;
        }
    } else {
#pragma unroll 1
        for (int j = 0; j < 16; ++j) {
            float u = x[0];
#pragma unroll
            for (int i = 1; i < 16; ++i) u = i == j ? x[i] : u;
            unsigned c;
            float dist;
            if (LEVELS == 3) {
                const float a = u - s.heap[1], b = u - s.heap[2];
                c = ((a > 0.0f) + (b > 0.0f) - 1) & 3;
                dist = fminf(fabsf(a), fabsf(b));
            } else {
                unsigned k = 1;
                dist = 4.0f;
#pragma unroll 1
                for (int l = 0; l < W; ++l) {
                    const float d = u - s.heap[k];
                    dist = fminf(dist, fabsf(d));
                    k = 2 * k + (d > 0.0f);
                }
                c = k - LEVELS;
            }
            if (j < 8) word[0] |= c << (j * W);
            else word[1] |= c << ((j - 8) * W);
            near |= (unsigned)(dist <= s.near) << j;
        }
    }
    uint64_t codes = word[0] | (uint64_t)word[1] << (8 * W);
    __half norm = __float2half_rn(n);
    bool wild = n2 < 1e-30f || n2 > 1e30f;  // a sum of squares that fp32 may not hold
    if (__any_sync(0xFFFFFFFFu, wild)) {
        // a group of zeros is decided as it stands (every coordinate is exactly zero); else every coordinate again. Where the sum
        // of squares is too large, the coordinates above are zeros of an infinite scale and say nothing
        bool nonzero = false;
#pragma unroll
        for (int j = 0; j < 16; ++j) nonzero |= !(x[j] == 0.0f);
        nonzero = __ballot_sync(0xFFFFFFFFu, nonzero) >> (lane & 24) & 0xFFu;
        if (wild) near = nonzero || n2 > 1e30f ? 0xFFFFu : 0u;
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
    extern __shared__ float2 s_table[];
    __shared__ int s_turn;
    const int tid = threadIdx.x, lane = tid & 31;
    for (int i = tid; i < 2 * kTable; i += kThreads) {
        const SideParams &s = p.side[i >= kTable];
        const int cell = (i >= kTable ? i - kTable : i) / kCopies;
        s_table[i] = make_float2(s.cell_mid[cell], __uint_as_float(s.cell_code[cell]));
    }
    if (tid == 0) s_turn = 0;
    __syncthreads();
    const long long all = p.side[0].warps + p.side[1].warps;
    // The block's tasks are handed out as its warps come for them: exact decisions make some of them much longer.
    for (;;) {
        int turn;
        if (lane == 0) turn = atomicAdd(&s_turn, 1);
        turn = __shfl_sync(0xFFFFFFFFu, turn, 0);
        const long long t = (long long)(turn >> 3) * gridDim.x * kWarps + (long long)blockIdx.x * kWarps + (turn & 7);
        if (t >= all) break;
        const int which = t >= p.side[0].warps;
        const SideParams &s = p.side[which];
        const long long task = which ? t - p.side[0].warps : t;
        const float2 *table = s_table + which * kTable;
        switch (s.bits) {
        case 2: encode<4, T>(p, s, table, task, lane); break;
        case 3: encode<8, T>(p, s, table, task, lane); break;
        case 4: encode<16, T>(p, s, table, task, lane); break;
        default: encode<3, T>(p, s, table, task, lane); break;
        }
    }
}

}  // namespace

// The cells of a codebook: an offset of the grid for which every cell has at most one midpoint and none lies within 1/64 of a
// cell of an edge (the cell of a coordinate is found to 1/128), looked for among 64. False if there is none.
static bool find_cells(const double *mid, int n, SideParams &s) {
    int at[15];
    for (int k = 0; k < 64; ++k) {
        const double offset = 65.0 + k / 64.0;  // -1 lies in cell 1, 1 in cell 130 at most
        bool ok = true;
        for (int l = 0; l < n && ok; ++l) {
            const double v = std::min(std::max(64.0 * mid[l] + offset, -1.5), kCells + 0.5);  // what no coordinate reaches: outside
            at[l] = (int)std::floor(v);
            const double in = v - at[l];
            if (at[l] >= 0 && at[l] < kCells) ok = in > 1.0 / 64 && in < 63.0 / 64 && (!l || at[l] != at[l - 1]);
        }
        if (!ok) continue;
        s.offset = (float)(65536.0 + offset);
        for (int c = 0, l = 0; c < kCells; ++c) {
            while (l < n && at[l] < c) ++l;  // midpoints below the cell
            s.cell_mid[c] = l < n && at[l] == c ? (float)mid[l] : 8.0f;  // 8: none here, and no coordinate is near it
            s.cell_code[c] = (uint8_t)l;
        }
        return true;
    }
    return false;
}

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
        double most = 0.0;  // the largest midpoint that a coordinate reaches
        for (int l = 0; l + 1 < levels; ++l) most = std::max(most, std::min(1.0, std::fabs(s.mid[l])));
        s.near = (float)(1.02 * std::ldexp(7.0 + 11.0 * most, -24));
        s.cells = find_cells(s.mid, levels - 1, s);
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
    const int grid = (int)std::min<long long>(blocks, 4LL * sm_count()), smem = 2 * kTable * (int)sizeof(float2);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == CQ_T_F32) kv_write_slots_kernel<float><<<grid, kThreads, smem, st>>>(p);
    else if (dtype == CQ_T_F16) kv_write_slots_kernel<__half><<<grid, kThreads, smem, st>>>(p);
    else kv_write_slots_kernel<__nv_bfloat16><<<grid, kThreads, smem, st>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return set_error(CQ_ERR_CUDA, "slot write launch: %s", cudaGetErrorString(e));
    return CQ_OK;
}

}  // namespace cq
