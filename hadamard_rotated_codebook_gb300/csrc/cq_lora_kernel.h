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
// Split. A piece is up to TOK tokens of one request. A cluster of C blocks takes a piece and a matrix: block c sums its c-th part of k for
// all ranks, its warps a part of that part each; the blocks' sums meet over distributed shared memory, added in block
// order by every block for itself; then block c does its c-th part of the outputs. One launch, no workspace, no
// atomics, and nothing depends on timing. What a block will read of B is asked for (into L2) before it begins with A.
//
// Precision. 16-bit and int8 activations meet the weights in one exact product each with fp32 sums. fp32 activations, and u in
// the second product, are two terms of 11 bits (tf32, which holds fp16 and bf16 weights exactly): what is lost is 2^-22.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdlib>
#include <type_traits>

#include "cq_layer.h"

namespace cq {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxCluster = 8;
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
// n of 4 consecutive weights of B.
__device__ __forceinline__ uint2 load_b(const uint16_t *p, int n, bool vec) {
    if (n <= 0) return make_uint2(0, 0);
    if (vec) {  // columns past an adapter's own rank may hold anything
        uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
        if (n < 4) v.y = n < 3 ? 0 : v.y & 0xFFFFu;
        if (n < 2) v.x &= 0xFFFFu;
        return v;
    }
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
struct Shape {
    static constexpr int kTok = 8 * NT * WT, kRank = 16 * MT, kParts = kWarps / WT;
    // row strides that keep the lanes of an access in different banks
    static constexpr int kPartRow = kRank + 4, kURow = MT == 1 ? 16 : kRank + 16;
    static constexpr int kSumBytes = kTok * kPartRow * 4, kUBytes = kTok * kURow * 4;
    static constexpr int kBlocks = NT > 1 || MT == 4 ? 2 : MT == 2 ? 3 : 4;  // on an SM
    static constexpr int kRoom = 228 * 1024 / kBlocks - 1024;
    // a warp's ring for the first product: 32 inputs a stage. What it holds is read before the sums take its place.
    static constexpr int kStage = 32 * (MT * 32 + NT * run_bytes<XK>());
    static constexpr int kDepth = kRoom / (kWarps * kStage) < 4 ? kRoom / (kWarps * kStage) : 4;
    static constexpr int kRing = kWarps * kDepth * kStage;
    // and one for y, a kilobyte a tile of 8 tokens and 32 outputs, behind the block's own sums (which others may still read)
    static constexpr int kDepthY = NT == 1 ? 0 : (kParts - 1) * kSumBytes > 48 * 1024 ? 6 : 4;
    static constexpr int kPartBytes = kParts * kSumBytes > kSumBytes + kDepthY * kWarps * 1024 ? kParts * kSumBytes : kSumBytes + kDepthY * kWarps * 1024;
    static constexpr int kSmem = kRing > kPartBytes + 2 * kUBytes ? kRing : kPartBytes + 2 * kUBytes;
    static_assert(kDepth >= 2 && kSmem <= kRoom, "shared memory");
};

template <typename T, int XK, int MT, int NT, int WT, bool VEC>
__global__ void __launch_bounds__(kThreads, (Shape<XK, MT, NT, WT>::kBlocks)) lora_kernel(const __grid_constant__ LoraParams p) {
    using S = Shape<XK, MT, NT, WT>;
    extern __shared__ __align__(16) float smem[];
    float *part = smem, *u_hi = smem + S::kPartBytes / 4, *u_lo = u_hi + S::kUBytes / 4;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int C = p.cluster, cta = C > 1 ? blockIdx.x % C : 0, mat = blockIdx.y;
    const float *y = p.d.y[mat];
    float *yo = p.d.y_out[mat];
    const Piece q = find_piece<S::kTok>(p, blockIdx.x / C, y == yo, lane, blockIdx.x + blockIdx.y + warp == 0);
    if (!q.n) return;  // the whole cluster
    const int out = p.d.out[mat], n_in = p.d.in;
    const int64_t yo_st = p.d.y_out_stride[mat];
    int64_t y_st = p.d.y_stride[mat];
    const int groups = (out + 31) / 32, g0 = (int)((long long)groups * cta / C), g1 = (int)((long long)groups * (cta + 1) / C);
    const uint16_t *B = static_cast<const uint16_t *>(p.d.b[mat]) + (int64_t)max(q.adapter, 0) * out * p.d.rank;
    if (q.rank && NT == 1) {  // few tokens: the weights are what takes time
        const uint8_t *from = reinterpret_cast<const uint8_t *>(B + (int64_t)g0 * 32 * p.d.rank);
        const int64_t bytes = ((int64_t)min(out, g1 * 32) - g0 * 32) * p.d.rank * 2;
        for (int64_t i = tid * 128ll; i < bytes; i += kThreads * 128ll) asm volatile("prefetch.global.L2 [%0];\n" ::"l"(from + i));
    }
    if (NT > 1 && p.vec_y[mat]) {  // many tokens: y
        const int w0 = g0 * 32, lines = (min(out, g1 * 32) - w0 + 31) / 32;
        for (int i = tid; i < q.n * lines; i += kThreads) {
            const int t = i / lines, l = i - t * lines;
            asm volatile("prefetch.global.L2 [%0];\n" ::"l"(y + (int64_t)(q.first + t) * y_st + w0 + l * 32));
        }
    }
    const float scale = q.rank && p.d.scales ? p.d.scales[q.adapter] : 1.0f;
    // Ranks in runs of kRank, each added to what the one before left (one run, nearly always).
#pragma unroll 1
    for (int r0 = 0; r0 == 0 || r0 < q.rank; r0 += S::kRank) {
        const int rank = min(S::kRank, q.rank - r0);
        if (rank > 0) {
            if (r0) {  // the other blocks have read this one's sums, and its warps u
                if (C > 1) asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
                __threadfence();  // copies will read what was stored
                __syncthreads();
            }
            // ------------------------------------------------ u: this warp's part of k --
            const int wk = warp / WT, wt = warp % WT;
            const int chunks = (n_in + 31) / 32, c0 = (int)((long long)chunks * cta / C), c1 = (int)((long long)chunks * (cta + 1) / C);
            const int live = min(NT, (q.n - wt * 8 * NT + 7) / 8);  // tiles with a token
            const uint16_t *A = static_cast<const uint16_t *>(p.d.a[mat]) + ((int64_t)q.adapter * p.d.rank + r0) * n_in;
            int64_t x_at[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) x_at[t] = (int64_t)(q.first + min(q.n - 1, (wt * NT + t) * 8 + g)) * p.d.x_stride;
            float acc[MT][NT][4];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[m][t][j] = 0.0f;
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
#pragma unroll
                for (int j = 0; j < S::kDepth - 1; ++j) send(c0 + wk + j * S::kParts, j);
            }
            int st = 0;
#pragma unroll 1
            for (int i = c0 + wk; i < c1; i += S::kParts) {
                const uint32_t from = ring + st * S::kStage;
                if (VEC) {
                    const int behind = st == 0 ? S::kDepth - 1 : st - 1;  // the stage read in the round before
                    send(i + (S::kDepth - 1) * S::kParts, behind);
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
            float *to = part + (size_t)wk * S::kTok * S::kPartRow;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (t >= live) break;
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int j = 0; j < 4; ++j) to[((wt * NT + t) * 8 + 2 * c + (j & 1)) * S::kPartRow + m * 16 + (j >> 1) * 8 + g] = acc[m][t][j];
            }
            __syncthreads();
            // ------------------------------------------- u: the warps' parts, then the blocks' --
            const int cells = (q.n + 7) / 8 * 8 * S::kRank;
            if (C > 1) {
                for (int i = tid; i < cells; i += kThreads) {
                    float *at = part + i / S::kRank * S::kPartRow + i % S::kRank, s = *at;
#pragma unroll
                    for (int k = 1; k < S::kParts; ++k) s += at[(size_t)k * S::kTok * S::kPartRow];
                    *at = s;
                }
                asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
            }
            for (int i = tid; i < cells; i += kThreads) {
                const int t = i / S::kRank, r = i % S::kRank;
                const float *at = part + t * S::kPartRow + r;
                float s = 0.0f;
                if (C > 1) {
                    const uint32_t here = smem_u32(at);
                    float v[kMaxCluster];  // all on their way before the first is added
#pragma unroll
                    for (int b = 0; b < kMaxCluster; ++b) {
                        v[b] = 0.0f;
                        if (b >= C) continue;
                        uint32_t there;
                        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(there) : "r"(here), "r"(b));
                        asm volatile("ld.shared::cluster.f32 %0, [%1];\n" : "=f"(v[b]) : "r"(there) : "memory");
                    }
#pragma unroll
                    for (int b = 0; b < kMaxCluster; ++b) s += v[b];
                } else {
                    s = *at;
#pragma unroll
                    for (int k = 1; k < S::kParts; ++k) s += at[(size_t)k * S::kTok * S::kPartRow];
                }
                if (XK == CQ_T_I8) s *= p.d.x_scale[q.first + min(t, q.n - 1)];
                uint32_t hi, lo;
                split(r < rank ? s * scale : 0.0f, hi, lo);  // ranks that are not there hold what x * 0 gave
                u_hi[t * S::kURow + r] = __uint_as_float(hi);
                u_lo[t * S::kURow + r] = __uint_as_float(lo);
            }
            if (C > 1) asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");  // this block has read the others
            __syncthreads();
        }
        // ---------------------------------------------------------- the outputs: 32 at a time --
        // Rows of a tile are dealt out so that a lane holds four consecutive outputs of two tokens.
        const bool vec_y = p.vec_y[mat];
        const int tiles = (q.n + 7) / 8, kts = (rank + 15) / 16, mine = g0 + warp < g1 ? (g1 - g0 - warp + kWarps - 1) / kWarps : 0;
        const uint32_t ring = smem_u32(smem) + S::kSumBytes + warp * S::kDepthY * 1024 + lane * 16;
        // A lane's elements of tile t of its j-th run of outputs are copied some tiles ahead of their turn.
        int sj = 0, stile = 0, sst = 0;
        auto send = [&]() {
            if (sj < mine) {
                const int o = (g0 + warp + sj * kWarps) * 32 + 4 * g;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int tok = stile * 8 + 2 * c + h;
                    const bool there = tok < q.n && o < out;
                    copy16(ring + sst * 1024 + h * 512, y + (there ? (int64_t)(q.first + tok) * y_st + o : 0), there);
                }
                if (++stile == tiles) stile = 0, ++sj;
            }
            copies_sent();
            if (++sst == S::kDepthY) sst = 0;
        };
        const bool ahead = NT > 1 && vec_y;
        if (ahead) {
#pragma unroll 1
            for (int j = 0; j < S::kDepthY - 1; ++j) send();
        }
        int st = 0;
#pragma unroll 1
        for (int j = 0; j < mine; ++j) {
            const int o = (g0 + warp + j * kWarps) * 32 + 4 * g, n_o = out - o;
            uint2 b[MT][4];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    b[m][i] = load_b(B + (int64_t)(o + i) * p.d.rank + r0 + m * 16 + 4 * c, i < n_o ? rank - m * 16 - 4 * c : 0, p.vec_b);
#pragma unroll 1
            for (int t = 0; t < tiles; ++t) {
                float v[2][4];
                if (ahead) {
                    send();
                    copies_landed<(S::kDepthY > 0 ? S::kDepthY - 1 : 0)>();
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int tok = t * 8 + 2 * c + h;
                    const float *from = y + (int64_t)(q.first + tok) * y_st + o;
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[h][i] = 0.0f;
                    if (ahead) {
                        const uint4 f = lds16(ring + st * 1024 + h * 512);
                        v[h][0] = __uint_as_float(f.x), v[h][1] = __uint_as_float(f.y), v[h][2] = __uint_as_float(f.z), v[h][3] = __uint_as_float(f.w);
                    } else if (tok < q.n && n_o > 0) {
                        if (vec_y) {
                            const float4 f = __ldcs(reinterpret_cast<const float4 *>(from));
                            v[h][0] = f.x, v[h][1] = f.y, v[h][2] = f.z, v[h][3] = f.w;
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (i < n_o) v[h][i] = from[i];
                        }
                    }
                }
                if (++st == S::kDepthY) st = 0;
                float d[2][4] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    if (m >= kts) break;
                    const int at = (t * 8 + g) * S::kURow + m * 16 + 4 * c;
                    const uint4 hi = *reinterpret_cast<const uint4 *>(u_hi + at), lo = *reinterpret_cast<const uint4 *>(u_lo + at);
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
        if (ahead) copies_landed<0>();
        y = yo, y_st = yo_st;
    }
    if (q.rank && C > 1) asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");  // no block ends while another reads its sums
}

// ---------------------------------------------------------------------- host --
template <typename T, int XK, int MT, int NT, int WT, bool VEC>
int launch_k(LoraParams &p, cudaStream_t st) {
    using S = Shape<XK, MT, NT, WT>;
    auto k = lora_kernel<T, XK, MT, NT, WT, VEC>;
    if (S::kSmem > 48 * 1024) {
        const int rc = ensure_smem(reinterpret_cast<const void *>(k), S::kSmem);
        if (rc) return rc;
    }
    const long long pieces = std::min<long long>(p.d.n_tokens, (long long)p.d.n_seqs + p.d.n_tokens / S::kTok);
    // Blocks of a cluster: parts of about 512 inputs or outputs, smaller ones where there are fewer than two blocks an SM.
    int widest = p.d.in;
    for (int j = 0; j < p.d.n_mats; ++j) widest = std::max(widest, p.d.out[j]);
    int C = 1;
    while (C < kMaxCluster && (widest > 512 * C || (widest > 128 * C && pieces * p.d.n_mats * C < 2 * sm_count()))) C *= 2;
    if (const char *e = getenv("LORA_C")) C = atoi(e);
    p.cluster = C;
    if (pieces * C > INT_MAX) return set_error(CQ_ERR_SHAPE, "%d tokens of %d requests are too many for one call", p.d.n_tokens, p.d.n_seqs);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(pieces * C), (unsigned)p.d.n_mats);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)C, at[0].val.clusterDim.y = 1, at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, k, p);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) {
        cudaGetLastError();
        return set_error(CQ_ERR_CUDA, "adapter launch: %s", cudaGetErrorString(e));
    }
    return CQ_OK;
}

// Tokens of a piece: 8 where requests have few, else as many as leave the sums of the first product in registers.
template <typename T, int XK, bool VEC>
int launch_x(LoraParams &p, cudaStream_t st) {
    const bool few = VEC && (long long)p.d.n_tokens <= 8ll * p.d.n_seqs;
    if (p.d.rank <= 16) return few ? launch_k<T, XK, 1, 1, 1, true>(p, st) : launch_k<T, XK, 1, XK == CQ_T_F32 ? 4 : 8, 2, VEC>(p, st);
    if (p.d.rank <= 32) return few ? launch_k<T, XK, 2, 1, 1, true>(p, st) : launch_k<T, XK, 2, 4, 2, VEC>(p, st);
    return few ? launch_k<T, XK, 4, 1, 1, true>(p, st) : launch_k<T, XK, 4, XK == CQ_T_F32 ? 2 : 4, 2, VEC>(p, st);
}
template <typename T>
int launch_t(LoraParams &p, bool vec, cudaStream_t st) {
    if (p.d.x_dtype == CQ_T_F32) return vec ? launch_x<T, CQ_T_F32, true>(p, st) : launch_x<T, CQ_T_F32, false>(p, st);
    if (p.d.x_dtype == CQ_T_I8) return vec ? launch_x<T, CQ_T_I8, true>(p, st) : launch_x<T, CQ_T_I8, false>(p, st);
    return vec ? launch_x<T, CQ_T_F16, true>(p, st) : launch_x<T, CQ_T_F16, false>(p, st);
}

}  // namespace
}  // namespace cq
