// cq_lora_kernel.h -- low-rank adapters of many requests, added to the outputs of shared projections.
//
//   u[t][r] = sum_k A[e][r][k] x[t][k],   y_out[t][o] = y[t][o] + scale[e] sum_r B[e][o][r] u[t][r],   e the adapter of t's request
//
// What bounds it is memory: a decode step reads each request's adapter once (2 rank (in + out) bytes), a prompt reads x and reads and
// writes y, while either product is a handful of operations a byte. Neither product fills a tensor core's tile: rank is the
// M side of the first (16 rows of A to a tile) and outputs are the M side of the second, tokens the N side in steps of 8, so that
// one token costs one narrow tile. mma.sync takes both operands from registers, which fit them as they come from memory:
// a lane loads 16 consecutive bytes of a row, and as both operands number their k the same way, any order of k will do. No
// tile is staged, no descriptor built.
//
// Split. A piece is up to TOK tokens of one request. The first kernel gives a piece and a matrix to `splits` blocks, each of
// which sums its part of k for all ranks (its warps a part of that part each) and leaves the sum in a workspace; the second
// gives runs of 32 outputs of a piece to warps, which add the parts in their order. No atomics, and nothing depends on
// timing. The second kernel begins while the first still runs: its blocks have found their pieces and have y and B on
// their way by the time the first one's sums are there.
//
// Precision. 16-bit and int8 activations meet the weights in one exact product each with fp32 sums. fp32 activations, and u in
// the second product, are two terms of 11 bits (tf32, which holds fp16 and bf16 weights exactly): what is lost is 2^-22.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <type_traits>

#include "cq_layer.h"

namespace cq {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kSeqs = 4;  // requests that a lane looks at in one go

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
template <typename T>
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if (std::is_same<T, __half>::value)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Half i of a register of two 16-bit weights as fp32.
template <typename T>
__device__ __forceinline__ uint32_t widen(uint32_t w, int i) {
    if (std::is_same<T, __nv_bfloat16>::value) return i ? w & 0xFFFF0000u : w << 16;
    return __float_as_uint(__half2float(__ushort_as_half((unsigned short)(i ? w >> 16 : w))));
}
// x as two terms of 11 bits. An infinity has no second term, and what is no number stays none.
__device__ __forceinline__ void split(float x, uint32_t &hi, uint32_t &lo) {
    hi = __float_as_uint(x) & 0xFFFFE000u;
    const float rest = fabsf(x) == INFINITY ? 0.0f : x - __uint_as_float(hi);
    asm("cvt.rna.tf32.f32 %0, %1;\n" : "=r"(lo) : "f"(rest));
}

// Eight consecutive activations, as the first product takes them: 16-bit pairs, or fp32.
template <int XK> struct XRun { uint32_t v[4]; };
template <> struct XRun<CQ_T_F32> { uint32_t v[8]; };

template <typename T>
__device__ __forceinline__ uint32_t pair_of(float x, float y) {
    if (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// XK: CQ_T_F32, CQ_T_I8, or 16 bits of the weights' own type (CQ_T_F16 stands for it).
template <int XK>
__host__ __device__ constexpr int run_bytes() { return XK == CQ_T_F32 ? 32 : XK == CQ_T_I8 ? 8 : 16; }
template <typename T>
__device__ __forceinline__ void pairs_of_i8(const uint32_t (&w)[2], uint32_t (&v)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t u = w[j / 2] >> (16 * (j & 1));
        v[j] = pair_of<T>((float)(int8_t)(u & 255u), (float)(int8_t)(u >> 8 & 255u));
    }
}
// n of the run's 8 elements, one by one.
template <typename T, int XK>
__device__ __forceinline__ XRun<XK> load_x(const void *x, int64_t at, int n) {
    XRun<XK> r = {};
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (j >= n) continue;
        if (XK == CQ_T_F32) r.v[XK == CQ_T_F32 ? j : 0] = __float_as_uint(__ldg(static_cast<const float *>(x) + at + j));
        else if (XK == CQ_T_I8) w[j / 4] |= (uint32_t)(uint8_t)__ldg(static_cast<const int8_t *>(x) + at + j) << (8 * (j & 3));
        else r.v[j / 2] |= (uint32_t)__ldg(static_cast<const uint16_t *>(x) + at + j) << (16 * (j & 1));
    }
    if (XK == CQ_T_I8) pairs_of_i8<T>(w, reinterpret_cast<uint32_t (&)[4]>(r.v));
    return r;
}
// Asynchronous copies of a lane's own runs into its own places of shared memory: nobody else reads them, so that the lane's own wait is
// all they need. A run that is not there becomes zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void *src, bool there) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;\n" ::"r"(dst), "l"(src), "r"(there ? 8 : 0) : "memory");
}
__device__ __forceinline__ void copies_sent() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_landed() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory"); }
__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];\n" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}
// Places of a run: 512 (or 256) bytes for a warp's 32 lanes, two such rows for fp32.
template <int XK>
__device__ __forceinline__ void send_x(uint32_t dst, int lane, const void *x, int64_t at, bool there) {
    const uint8_t *from = static_cast<const uint8_t *>(x) + (there ? at * (run_bytes<XK>() / 8) : 0);
    if (XK == CQ_T_I8) {
        copy8(dst + lane * 8, from, there);
    } else {
        copy16(dst + lane * 16, from, there);
        if (XK == CQ_T_F32) copy16(dst + 512 + lane * 16, from + 16, there);
    }
}
template <typename T, int XK>
__device__ __forceinline__ XRun<XK> take_x(uint32_t src, int lane) {
    XRun<XK> r = {};
    if (XK == CQ_T_I8) {
        const uint2 w = lds8(src + lane * 8);
        const uint32_t u[2] = {w.x, w.y};
        pairs_of_i8<T>(u, reinterpret_cast<uint32_t (&)[4]>(r.v));
    } else {
        const uint4 a = lds16(src + lane * 16);
        r.v[0] = a.x, r.v[1] = a.y, r.v[2] = a.z, r.v[3] = a.w;
        if (XK == CQ_T_F32) {
            const uint4 b = lds16(src + 512 + lane * 16);
            constexpr int o = XK == CQ_T_F32 ? 4 : 0;
            r.v[o] = b.x, r.v[o + 1] = b.y, r.v[o + 2] = b.z, r.v[o + 3] = b.w;
        }
    }
    return r;
}
// n of 8 consecutive weights of A.
__device__ __forceinline__ uint4 load_a(const uint16_t *p, int n) {
    uint32_t v[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < n) v[j / 2] |= (uint32_t)__ldg(p + j) << (16 * (j & 1));
    return make_uint4(v[0], v[1], v[2], v[3]);
}
// The first n of 4 consecutive weights of B: columns past an adapter's own rank may hold anything.
__device__ __forceinline__ uint2 cut_b(uint2 v, int n) {
    if (n < 4) v.y = n < 3 ? 0 : v.y & 0xFFFFu;
    if (n < 2) v.x = n < 1 ? 0 : v.x & 0xFFFFu;
    return v;
}
__device__ __forceinline__ uint2 load_b(const uint16_t *p, int n, bool vec) {
    if (n <= 0) return make_uint2(0, 0);
    if (vec) return cut_b(__ldg(reinterpret_cast<const uint2 *>(p)), n);
    uint32_t v[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j < n) v[j / 2] |= (uint32_t)__ldg(p + j) << (16 * (j & 1));
    return make_uint2(v[0], v[1]);
}

struct Piece {
    int first, n, adapter, rank;  // tokens first .. first + n - 1; adapter -1: none
};
// The request s, cut to what the sizes allow; `bad` where it does not fit them.
__device__ __forceinline__ Piece seq_at(const LoraParams &p, int s, bool &bad) {
    Piece q;
    const int a = p.d.cu_tokens[s], b = p.d.cu_tokens[s + 1];
    const bool out = a < 0 || b < a || b > p.d.n_tokens;
    q.first = a, q.n = out ? 0 : b - a, q.adapter = p.d.adapters[s], q.rank = 0;
    bad |= out;
    if (q.adapter < 0 || q.adapter >= p.d.n_adapters) {
        bad |= q.adapter != -1;
        q.adapter = -1;
    }
    return q;
}
// The piece-th piece of up to TOK tokens over all requests (those without an adapter have none where `skip`); n = 0 past the last.
// Every warp finds it for itself.
template <int TOK>
__device__ Piece find_piece(const LoraParams &p, int piece, bool skip, int lane, bool report) {
    Piece q = {};
    bool bad = false;
    int before = 0;
#pragma unroll 1
    for (int base = 0; base < p.d.n_seqs; base += 32 * kSeqs) {
        Piece mine[kSeqs];
        int count[kSeqs], sum = 0;
#pragma unroll
        for (int i = 0; i < kSeqs; ++i) {
            const int s = base + lane * kSeqs + i;
            mine[i] = {};
            if (s < p.d.n_seqs) mine[i] = seq_at(p, s, bad);
            count[i] = skip && mine[i].adapter < 0 ? 0 : (int)(((long long)mine[i].n + TOK - 1) / TOK);
            sum += count[i];
        }
        int upto = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
            if (lane >= o) upto += v;
        }
        const int all = __shfl_sync(0xFFFFFFFFu, upto, 31);
        if (!q.n && piece - before < all) {  // uniform
            int at = piece - before - (upto - sum);
            const bool here = at >= 0 && at < sum;
            if (here) {
#pragma unroll
                for (int i = 0; i < kSeqs; ++i) {
                    if (at >= 0 && at < count[i]) {
                        q = mine[i];
                        q.first += at * TOK;
                        q.n = min(TOK, q.n - at * TOK);
                    }
                    at -= count[i];
                }
            }
            const int src = __ffs(__ballot_sync(0xFFFFFFFFu, here)) - 1;
            q.first = __shfl_sync(0xFFFFFFFFu, q.first, src);
            q.n = __shfl_sync(0xFFFFFFFFu, q.n, src);
            q.adapter = __shfl_sync(0xFFFFFFFFu, q.adapter, src);
            if (!report) break;
        }
        before += all;
    }
    if (report && __any_sync(0xFFFFFFFFu, bad) && lane == 0) atomicOr(p.status, kStatusIndex);
    q.rank = p.d.rank;
    if (q.n && q.adapter >= 0 && p.d.ranks) {
        q.rank = p.d.ranks[q.adapter];
        if (q.rank < 0 || q.rank > p.d.rank) {
            if (lane == 0) atomicOr(p.status, kStatusIndex);
            q.adapter = -1;
        }
    }
    if (q.adapter < 0) q.rank = 0;
    return q;
}

// MT: tiles of 16 ranks; NT: tiles of 8 tokens of a warp; WT: warps side by side along the tokens (the others split k).
template <int XK, int MT, int NT, int WT>
struct Down {
    static constexpr int kTok = 8 * NT * WT, kRank = 16 * MT, kParts = kWarps / WT;
    static constexpr int kRow = kRank + 4;  // keeps the lanes that write a sum in different banks
    static constexpr int kBlocks = NT > 1 || MT == 4 ? 2 : 3;  // on an SM
    static constexpr int kRoom = 228 * 1024 / kBlocks - 1024;
    // a warp's ring: 32 inputs a stage. What it holds is read before the sums take its place.
    static constexpr int kStage = 32 * (MT * 32 + NT * run_bytes<XK>());
    static constexpr int kDepth = kRoom / (kWarps * kStage) < 6 ? kRoom / (kWarps * kStage) : 6;
    static constexpr int kRing = kWarps * kDepth * kStage, kSums = kParts * kTok * kRow * 4;
    static constexpr int kSmem = kRing > kSums ? kRing : kSums;
    static_assert(kDepth >= 2 && kSmem <= kRoom, "shared memory");
};

// u[t][r] over a part of k: the blocks of a piece and matrix write parts of their own (p.u: [matrix][part][token][p.u_row]).
template <typename T, int XK, int MT, int NT, int WT, bool VEC>
__global__ void __launch_bounds__(kThreads, (Down<XK, MT, NT, WT>::kBlocks)) lora_down_kernel(const __grid_constant__ LoraParams p) {
    using S = Down<XK, MT, NT, WT>;
    extern __shared__ __align__(16) float smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int cut = blockIdx.x % p.splits, mat = blockIdx.y, r0 = blockIdx.z * S::kRank;
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const Piece q = find_piece<S::kTok>(p, blockIdx.x / p.splits, true, lane, blockIdx.x + blockIdx.y + blockIdx.z + warp == 0);
    const int rank = min(S::kRank, q.rank - r0), n_in = p.d.in;
    if (!q.n || rank <= 0) return;
    const int wk = warp / WT, wt = warp % WT;
    const int chunks = (n_in + 31) / 32, c0 = (int)((long long)chunks * cut / p.splits), c1 = (int)((long long)chunks * (cut + 1) / p.splits);
    const int live = min(NT, (q.n - wt * 8 * NT + 7) / 8);  // tiles with a token
    const uint16_t *A = static_cast<const uint16_t *>(p.d.a[mat]) + ((int64_t)q.adapter * p.d.rank + r0) * n_in;
    int64_t x_at[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) x_at[t] = (int64_t)(q.first + min(q.n - 1, (wt * NT + t) * 8 + g)) * p.d.x_stride;
    const uint32_t ring = smem_u32(smem) + warp * S::kDepth * S::kStage;
    auto send = [&](int i, int st) {
        const int k = i * 32 + c * 8;
        const uint32_t to = ring + st * S::kStage;
        if (i < c1) {
#pragma unroll
            for (int h = 0; h < 2 * MT; ++h) {
                const int r = h * 8 + g;
                const bool there = r < rank && k < n_in;
                copy16(to + h * 512 + lane * 16, A + (there ? (int64_t)r * n_in + k : 0), there);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t)
                if (t < live) send_x<XK>(to + MT * 1024 + t * 32 * run_bytes<XK>(), lane, p.d.x, x_at[t] + k, k < n_in);
        }
        copies_sent();
    };
    if (VEC) {
#pragma unroll 1
        for (int j = 0; j < S::kDepth - 1; ++j) send(c0 + wk + j * S::kParts, j);
    }
    const float scale = p.d.scales ? p.d.scales[q.adapter] : 1.0f;
    float acc[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[m][t][j] = 0.0f;
    int st = 0;
#pragma unroll 1
    for (int i = c0 + wk; i < c1; i += S::kParts) {
        const uint32_t from = ring + st * S::kStage;
        if (VEC) {
            send(i + (S::kDepth - 1) * S::kParts, st == 0 ? S::kDepth - 1 : st - 1);  // where the round before was read
            copies_landed<S::kDepth - 1>();
            if (++st == S::kDepth) st = 0;
        }
        const int k = i * 32 + c * 8, n = n_in - k;
        XRun<XK> x[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (t >= live) break;
            if (VEC) x[t] = take_x<T, XK>(from + MT * 1024 + t * 32 * run_bytes<XK>(), lane);
            else x[t] = load_x<T, XK>(p.d.x, x_at[t] + k, n);
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            uint4 a[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = m * 16 + h * 8 + g;
                if (VEC) a[h] = lds16(from + (2 * m + h) * 512 + lane * 16);
                else a[h] = load_a(A + (int64_t)r * n_in + k, r < rank ? n : 0);
            }
            const uint32_t lo[4] = {a[0].x, a[0].y, a[0].z, a[0].w}, hi[4] = {a[1].x, a[1].y, a[1].z, a[1].w};
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (t >= live) break;
                if (XK == CQ_T_F32) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t h0, l0, h1, l1;
                        split(__uint_as_float(x[t].v[XK == CQ_T_F32 ? 2 * j : 0]), h0, l0);
                        split(__uint_as_float(x[t].v[XK == CQ_T_F32 ? 2 * j + 1 : 0]), h1, l1);
                        const uint32_t a0 = widen<T>(lo[j], 0), a1 = widen<T>(hi[j], 0), a2 = widen<T>(lo[j], 1), a3 = widen<T>(hi[j], 1);
                        mma_tf32(acc[m][t], a0, a1, a2, a3, l0, l1);
                        mma_tf32(acc[m][t], a0, a1, a2, a3, h0, h1);
                    }
                } else {
                    mma16<T>(acc[m][t], lo[0], hi[0], lo[1], hi[1], x[t].v[0], x[t].v[1]);
                    mma16<T>(acc[m][t], lo[2], hi[2], lo[3], hi[3], x[t].v[2], x[t].v[3]);
                }
            }
        }
    }
    if (VEC) {
        copies_landed<0>();
        __syncthreads();  // the sums take the rings' place
    }
    float *to = smem + (size_t)wk * S::kTok * S::kRow;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        if (t >= live) break;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j) to[((wt * NT + t) * 8 + 2 * c + (j & 1)) * S::kRow + m * 16 + (j >> 1) * 8 + g] = acc[m][t][j];
    }
    __syncthreads();
    float *u = p.u + (((int64_t)mat * p.splits + cut) * p.d.n_tokens + q.first) * p.u_row + r0;
    for (int i = tid; i < q.n * S::kRank; i += kThreads) {
        const int t = i / S::kRank, r = i % S::kRank;
        const float *at = smem + t * S::kRow + r;
        float s = *at;
#pragma unroll
        for (int k = 1; k < S::kParts; ++k) s += at[(size_t)k * S::kTok * S::kRow];
        if (XK == CQ_T_I8) s *= p.d.x_scale[q.first + t];
        u[(int64_t)t * p.u_row + r] = r < rank ? s * scale : 0.0f;  // ranks that are not there hold what x * 0 gave
    }
}

// TOK: tokens of a piece, a multiple of 8. FEW: 8 tokens, and B comes through the ring too.
template <int MT, int TOK, bool FEW>
struct Up {
    static constexpr int kRank = 16 * MT;
    static constexpr int kRow = MT == 1 ? 16 : kRank + 16;  // rows of u that keep the lanes which read them in different banks
    static constexpr int kU = TOK * kRow * 4;
    static constexpr int kBlocks = MT == 4 ? 2 : 3;
    // a warp's ring: a kilobyte of y (8 tokens, 32 outputs) a stage, and MT of B where there is a run of outputs to each
    static constexpr int kStage = 1024 + (FEW ? MT * 1024 : 0), kDepth = FEW ? MT == 4 ? 2 : 3 : 5;
    static constexpr int kSmem = 2 * kU + kWarps * kDepth * kStage;
    static_assert(kSmem <= 228 * 1024 / kBlocks - 1024, "shared memory");
};

// y_out = y + B u over runs of 32 outputs: a block's warps take p.runs of them after another.
template <typename T, int MT, int TOK, bool FEW>
__global__ void __launch_bounds__(kThreads, (Up<MT, TOK, FEW>::kBlocks)) lora_up_kernel(const __grid_constant__ LoraParams p) {
    using S = Up<MT, TOK, FEW>;
    extern __shared__ __align__(16) float smem[];
    float *u_hi = smem, *u_lo = smem + S::kU / 4;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3, mat = blockIdx.z;
    const float *y = p.d.y[mat];
    float *yo = p.d.y_out[mat];
    const int out = p.d.out[mat], groups = (out + 31) / 32, g0 = blockIdx.y * p.runs * kWarps + warp, g1 = min(groups, ((int)blockIdx.y + 1) * p.runs * kWarps);
    const Piece q = (int)blockIdx.y * p.runs * kWarps < groups ? find_piece<TOK>(p, blockIdx.x, y == yo, lane, false) : Piece{};
    if (!q.n) {
        asm volatile("griddepcontrol.wait;\n" ::: "memory");  // every block: what follows this kernel also follows the one before it
        return;
    }
    const int64_t yo_st = p.d.y_out_stride[mat];
    int64_t y_st = p.d.y_stride[mat];
    const uint16_t *B = static_cast<const uint16_t *>(p.d.b[mat]) + (int64_t)max(q.adapter, 0) * out * p.d.rank;
    const bool vec_y = p.vec_y[mat], ring_b = FEW && p.vec_b;
    const int tiles = (q.n + 7) / 8, mine = g0 < g1 ? (g1 - g0 + kWarps - 1) / kWarps : 0;
    const uint32_t ring = smem_u32(smem) + 2 * S::kU + warp * S::kDepth * S::kStage;
    // Ranks in runs of kRank, each added to what the one before left (one run, nearly always).
#pragma unroll 1
    for (int r0 = 0; r0 == 0 || r0 < q.rank; r0 += S::kRank) {
        const int rank = min(S::kRank, q.rank - r0);
        // A lane's elements of tile t of its j-th run of outputs are copied some tiles ahead of their turn.
        int sj = 0, stile = 0, sst = 0;
        auto send = [&]() {
            if (sj < mine) {
                const int o = (g0 + sj * kWarps) * 32 + 4 * g;
                const uint32_t to = ring + sst * S::kStage;
                if (vec_y) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int tok = stile * 8 + 2 * c + h;
                        const bool there = tok < q.n && o < out;
                        copy16(to + h * 512 + lane * 16, y + (there ? (int64_t)(q.first + tok) * y_st + o : 0), there);
                    }
                }
                if (ring_b) {
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const bool there = o + i < out && m * 16 + 4 * c < rank;
                            copy8(to + 1024 + (m * 4 + i) * 256 + lane * 8, B + (there ? (int64_t)(o + i) * p.d.rank + r0 + m * 16 + 4 * c : 0), there);
                        }
                }
                if (++stile == tiles) stile = 0, ++sj;
            }
            copies_sent();
            if (++sst == S::kDepth) sst = 0;
        };
#pragma unroll 1
        for (int j = 0; j < S::kDepth - 1; ++j) send();
        if (r0) __syncthreads();  // u is read
        else asm volatile("griddepcontrol.wait;\n" ::: "memory");
        // ------------------------------------------------------------- u as two terms --
        if (rank > 0) {
            const float *from = p.u + ((int64_t)mat * p.splits * p.d.n_tokens + q.first) * p.u_row + r0;
            const int64_t next = (int64_t)p.d.n_tokens * p.u_row;
            for (int i = tid; i < tiles * 8 * (S::kRank / 4); i += kThreads) {
                const int t = i / (S::kRank / 4), r = i % (S::kRank / 4) * 4;
                float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (t < q.n) {
                    float4 v[kMaxSplits];  // all on their way before the first is added
#pragma unroll
                    for (int k = 0; k < kMaxSplits; ++k) {
                        v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        if (k < p.splits) v[k] = __ldcg(reinterpret_cast<const float4 *>(from + k * next + (int64_t)t * p.u_row + r));
                    }
#pragma unroll
                    for (int k = 0; k < kMaxSplits; ++k) s.x += v[k].x, s.y += v[k].y, s.z += v[k].z, s.w += v[k].w;
                }
                uint4 hi, lo;
                split(s.x, hi.x, lo.x), split(s.y, hi.y, lo.y), split(s.z, hi.z, lo.z), split(s.w, hi.w, lo.w);
                *reinterpret_cast<uint4 *>(u_hi + t * S::kRow + r) = hi;
                *reinterpret_cast<uint4 *>(u_lo + t * S::kRow + r) = lo;
            }
            __syncthreads();
        }
        // ---------------------------------------------------------- the outputs: 32 at a time --
        // Rows of a tile are dealt out so that a lane holds four consecutive outputs of two tokens.
        const int kts = (rank + 15) / 16;
        int st = 0;
#pragma unroll 1
        for (int j = 0; j < mine; ++j) {
            const int o = (g0 + j * kWarps) * 32 + 4 * g, n_o = out - o;
            uint2 b[MT][4];
            if (!ring_b) {
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        b[m][i] = load_b(B + (int64_t)(o + i) * p.d.rank + r0 + m * 16 + 4 * c, i < n_o ? rank - m * 16 - 4 * c : 0, p.vec_b);
            }
#pragma unroll 1
            for (int t = 0; t < tiles; ++t) {
                send();
                copies_landed<S::kDepth - 1>();
                const uint32_t at = ring + st * S::kStage;
                if (++st == S::kDepth) st = 0;
                if (ring_b) {
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int i = 0; i < 4; ++i) b[m][i] = cut_b(lds8(at + 1024 + (m * 4 + i) * 256 + lane * 8), rank - m * 16 - 4 * c);
                }
                float v[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int tok = t * 8 + 2 * c + h;
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[h][i] = 0.0f;
                    if (vec_y) {
                        const uint4 f = lds16(at + h * 512 + lane * 16);
                        v[h][0] = __uint_as_float(f.x), v[h][1] = __uint_as_float(f.y), v[h][2] = __uint_as_float(f.z), v[h][3] = __uint_as_float(f.w);
                    } else if (tok < q.n) {
                        const float *from = y + (int64_t)(q.first + tok) * y_st + o;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (i < n_o) v[h][i] = from[i];
                    }
                }
                float d[2][4] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    if (m >= kts) break;
                    const int row = (t * 8 + g) * S::kRow + m * 16 + 4 * c;
                    const uint4 hi = *reinterpret_cast<const uint4 *>(u_hi + row), lo = *reinterpret_cast<const uint4 *>(u_lo + row);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t h0 = k ? hi.z : hi.x, h1 = k ? hi.w : hi.y, l0 = k ? lo.z : lo.x, l1 = k ? lo.w : lo.y;
#pragma unroll
                        for (int f = 0; f < 2; ++f) {
                            const uint32_t w0 = k ? b[m][2 * f].y : b[m][2 * f].x, w1 = k ? b[m][2 * f + 1].y : b[m][2 * f + 1].x;
                            const uint32_t a0 = widen<T>(w0, 0), a1 = widen<T>(w1, 0), a2 = widen<T>(w0, 1), a3 = widen<T>(w1, 1);
                            mma_tf32(d[f], a0, a1, a2, a3, l0, l1);
                            mma_tf32(d[f], a0, a1, a2, a3, h0, h1);
                        }
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int tok = t * 8 + 2 * c + h;
                    if (tok >= q.n || n_o <= 0) continue;
                    if (rank > 0) v[h][0] += d[0][h], v[h][1] += d[0][2 + h], v[h][2] += d[1][h], v[h][3] += d[1][2 + h];
                    float *to = yo + (int64_t)(q.first + tok) * yo_st + o;
                    if (vec_y) {
                        *reinterpret_cast<float4 *>(to) = make_float4(v[h][0], v[h][1], v[h][2], v[h][3]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (i < n_o) to[i] = v[h][i];
                    }
                }
            }
        }
        copies_landed<0>();
        if (r0 + S::kRank < q.rank) __threadfence();  // copies will read what was stored
        y = yo, y_st = yo_st;
    }
}

// ---------------------------------------------------------------------- host --
template <typename T, int XK, int MT, int NT, int WT, bool VEC>
int launch_down(const LoraParams &p, cudaStream_t st) {
    using S = Down<XK, MT, NT, WT>;
    auto k = lora_down_kernel<T, XK, MT, NT, WT, VEC>;
    if (S::kSmem > 48 * 1024) {
        const int rc = ensure_smem(reinterpret_cast<const void *>(k), S::kSmem);
        if (rc) return rc;
    }
    k<<<dim3(p.pieces * p.splits, p.d.n_mats, p.u_row / S::kRank), kThreads, S::kSmem, st>>>(p);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? CQ_OK : set_error(CQ_ERR_CUDA, "adapter launch: %s", cudaGetErrorString(e));
}
template <typename T, int MT, int TOK, bool FEW>
int launch_up(LoraParams &p, cudaStream_t st) {
    using S = Up<MT, TOK, FEW>;
    auto k = lora_up_kernel<T, MT, TOK, FEW>;
    if (S::kSmem > 48 * 1024) {
        const int rc = ensure_smem(reinterpret_cast<const void *>(k), S::kSmem);
        if (rc) return rc;
    }
    int groups = 1;
    for (int j = 0; j < p.d.n_mats; ++j) groups = std::max(groups, (p.d.out[j] + 31) / 32);
    // Runs of outputs of a warp: one, and more while that leaves every SM four blocks.
    p.runs = 1;
    while (p.runs < 8 && (long long)p.pieces * p.d.n_mats * ((groups + 2 * kWarps * p.runs - 1) / (2 * kWarps * p.runs)) >= 4ll * sm_count()) p.runs *= 2;
    const int rows = (groups + kWarps * p.runs - 1) / (kWarps * p.runs);
    if (rows > 65535) return set_error(CQ_ERR_SHAPE, "%d outputs are too many", groups * 32);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.pieces, (unsigned)rows, (unsigned)p.d.n_mats);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, k, p);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e == cudaSuccess) return CQ_OK;
    cudaGetLastError();
    return set_error(CQ_ERR_CUDA, "adapter launch: %s", cudaGetErrorString(e));
}

template <typename T, int XK, int MT, bool VEC>
int launch_r(LoraParams &p, cudaStream_t st) {
    constexpr int WT = lora_warps_along(false), NT = lora_tokens(XK, MT, false) / (8 * WT);
    int rc;
    if (VEC && p.few) rc = launch_down<T, XK, MT, 1, 1, true>(p, st);
    else rc = launch_down<T, XK, MT, NT, WT, VEC>(p, st);
    if (rc) return rc;
    return p.few ? launch_up<T, MT, 8, true>(p, st) : launch_up<T, MT, 8 * NT * WT, false>(p, st);
}
template <typename T, int XK, bool VEC>
int launch_x(LoraParams &p, cudaStream_t st) {
    switch (lora_rank_tiles(p.d.rank)) {
    case 1: return launch_r<T, XK, 1, VEC>(p, st);
    case 2: return launch_r<T, XK, 2, VEC>(p, st);
    default: return launch_r<T, XK, 4, VEC>(p, st);
    }
}
template <typename T>
int launch_t(LoraParams &p, cudaStream_t st) {
    if (p.d.x_dtype == CQ_T_F32) return p.vec ? launch_x<T, CQ_T_F32, true>(p, st) : launch_x<T, CQ_T_F32, false>(p, st);
    if (p.d.x_dtype == CQ_T_I8) return p.vec ? launch_x<T, CQ_T_I8, true>(p, st) : launch_x<T, CQ_T_I8, false>(p, st);
    return p.vec ? launch_x<T, CQ_T_F16, true>(p, st) : launch_x<T, CQ_T_F16, false>(p, st);
}

}  // namespace
}  // namespace cq
