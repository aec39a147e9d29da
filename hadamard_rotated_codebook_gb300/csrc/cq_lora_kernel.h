// cq_lora_kernel.h -- low-rank adapters of many requests, added to the outputs of shared projections.
//
//   u[t][r] = sum_k A[e][r][k] x[t][k],   y_out[t][o] = y[t][o] + scale[e] sum_r B[e][o][r] u[t][r],   e the adapter of t's request
//
// What bounds it is memory: a decode step reads each request's adapter once (2 rank (in + out) bytes), a prompt reads x and reads and
// writes y, while either product is a handful of operations a byte.
//
// Split. A piece is up to so many tokens of one request. The first kernel gives a piece and a matrix to `splits` blocks, each of
// which sums its part of k for all ranks and leaves the sum in a workspace; the second gives tiles of outputs to blocks, which
// add the parts in their order. No atomics on values, and nothing depends on timing. The second kernel begins while the first still
// runs: its blocks have found their pieces and have y and B on their way by the time the first one's sums are there. (One kernel
// of clusters that met over distributed shared memory took 32 us for 64 decodes where the two take 16, and 211 us for the
// prompt below: a cluster's barriers stand between its loads.)
//
// Few tokens a request (lora_down_kernel, lora_up_kernel): pieces of 8 on mma.sync. Rank is the M side of the first product (16 rows of A to a
// tile), outputs are the M side of the second, tokens the N side, so that one token costs one narrow tile; tcgen05's least tile is
// 128 rows. A lane copies 16 consecutive bytes of a row, and as both operands number their k the same way, any order of k will
// do: what it copied is what it needs, and its own wait is all the synchronisation there is.
// Many tokens (lora_down_many_kernel, lora_up_many_kernel): tcgen05, fed by tensor copies. Tokens are the M side of the first product and
// outputs of the second, see there. Rows that tensor copies cannot reach and fp32 activations take lora_down_kernel in larger pieces.
//
// Precision. 16-bit and int8 activations meet the weights in one exact product each with fp32 sums. fp32 activations are two
// terms of 11 bits (tf32, which holds fp16 and bf16 weights exactly): what is lost is 2^-22. u, summed in fp32, is three
// terms of bf16 or two of fp16 (Terms).
//
// Measured: 64 decodes with 60 adapters, 4096 to 4096, 1024 and 1024, rank 16, int8 (38.8 MB): 16 us, 2.4 TB/s or 36% of the copy rate, 5.7 us
// being the floor: memory's latency twice in a row and the launch, with issue slots at half; 256 decodes 45 us, 53%. A prompt of 8190
// tokens of three requests, 4096 to 4096, rank 64, bf16 (339 MB): 67 us, 75%, floor 50; rank 16, int8: 61 us, 73%. One token, 512 to
// 512, 256 and 256, rank 8: 5 us, two kernels' latency.
// Tried and slower for prompts: mma.sync in both (97 to 146 us: 1.4 instructions an element), y in rows of 512 bytes by plain bulk copies (125 us: a
// copy of any size costs the copy engine as much), y loaded by the threads that add (124 us).
#pragma once

#include <cuda.h>
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
constexpr unsigned kSpin = 1u << 20;
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
// (One warp.)
template <int TOK>
__device__ Piece search_piece(const LoraParams &p, int piece, bool skip, int lane, bool report) {
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

// Likewise, for a whole block.
template <int TOK>
__device__ __forceinline__ Piece find_piece(const LoraParams &p, int piece, bool skip, int warp, int lane, bool report) {
    __shared__ Piece found;
    if (warp == 0) {
        const Piece q = search_piece<TOK>(p, piece, skip, lane, report);
        if (lane == 0) found = q;
    }
    __syncthreads();
    Piece q;  // through a shuffle: the compiler would read shared memory again wherever they are used
    q.first = __shfl_sync(0xFFFFFFFFu, found.first, 0), q.n = __shfl_sync(0xFFFFFFFFu, found.n, 0);
    q.adapter = __shfl_sync(0xFFFFFFFFu, found.adapter, 0), q.rank = __shfl_sync(0xFFFFFFFFu, found.rank, 0);
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
    const Piece q = search_piece<S::kTok>(p, blockIdx.x / p.splits, true, lane, blockIdx.x + blockIdx.y + blockIdx.z + warp == 0);
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

// u as the second product takes it, in terms of the weights' type: three of bf16 (24 bits together); two of fp16 (22), where a token's
// values are first multiplied by the power of two that brings its largest to 2^13..2^14, so that no term leaves fp16.
template <typename T> struct Terms { static constexpr int n = std::is_same<T, __half>::value ? 2 : 3; };
template <typename T>
__device__ __forceinline__ float term_of(float x) {
    return std::is_same<T, __half>::value ? __half2float(__float2half_rn(x)) : __bfloat162float(__float2bfloat16_rn(x));
}
// The next term of four values, and what it leaves of them (of an infinity, and of what rounds to one, nothing; what is no number stays none).
template <typename T>
__device__ __forceinline__ uint2 next_term(float (&x)[4]) {
    float t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        t[i] = term_of<T>(x[i]);
        x[i] = fabsf(t[i]) == INFINITY ? 0.0f : x[i] - t[i];
    }
    return make_uint2(pair_of<T>(t[0], t[1]), pair_of<T>(t[2], t[3]));
}

// Magnitudes are ordered as integers; what is not finite scales nothing.
__device__ __forceinline__ uint32_t magnitude(float x) {
    const uint32_t m = __float_as_uint(x) & 0x7FFFFFFFu;
    return m < 0x7F800000u ? m : 0u;
}
// What takes the power of two that brings the largest magnitude to 2^13..2^14 out again. (Its reciprocal has the exponent 254 - its own.)
__device__ __forceinline__ float back_of(uint32_t top) { return __uint_as_float((uint32_t)(max(14, (int)(top >> 23)) - 13) << 23); }

// The parts' sums of a piece's `tokens` (zero past its end), ranks r0 .. r0 + RANK - 1, as terms: put(term, token, rank, four values). A
// token's power of two goes to back[token], or is there already (`scaled`). kThreads threads.
template <typename T, int RANK, typename Put>
__device__ __forceinline__ void gather_u(const LoraParams &p, const Piece &q, int mat, int r0, int tokens, float *back, bool scaled, Put put) {
    constexpr int kFours = RANK / 4;  // of a token; they lie side by side in a warp
    const float *from = p.u + ((int64_t)mat * p.splits * p.d.n_tokens + q.first) * p.u_row + r0;
    const int64_t next = (int64_t)p.d.n_tokens * p.u_row;
    const int cells = tokens * kFours;
    for (int base = 0; base < cells; base += 2 * kThreads) {
        float4 s[2] = {make_float4(0.0f, 0.0f, 0.0f, 0.0f), make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
        for (int k0 = 0; k0 < p.splits; k0 += 4) {
            float4 v[2][4];  // all on their way before the first is added
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int i = base + h * kThreads + (int)threadIdx.x, t = i / kFours, r = i % kFours * 4;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    v[h][k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (t < q.n && k0 + k < p.splits) v[h][k] = __ldcg(reinterpret_cast<const float4 *>(from + (k0 + k) * next + (int64_t)t * p.u_row + r));
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int k = 0; k < 4; ++k) s[h].x += v[h][k].x, s[h].y += v[h][k].y, s[h].z += v[h][k].z, s[h].w += v[h][k].w;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = base + h * kThreads + (int)threadIdx.x, t = i / kFours, r = i % kFours * 4;
            float x[4] = {s[h].x, s[h].y, s[h].z, s[h].w};
            if (std::is_same<T, __half>::value) {
                uint32_t top = max(max(magnitude(x[0]), magnitude(x[1])), max(magnitude(x[2]), magnitude(x[3])));
#pragma unroll
                for (int o = 1; o < kFours; o <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                float down = back_of(top);
                if (scaled && i < cells) down = back[t];
                else if (i < cells && r == 0) back[t] = down;
                const float up = __uint_as_float((254u << 23) - __float_as_uint(down));
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] *= up;
            }
            if (i >= cells) continue;
#pragma unroll
            for (int k = 0; k < Terms<T>::n; ++k) put(k, t, r, next_term<T>(x));
        }
    }
}

// The second product where requests have few tokens: pieces of 8.
template <typename T, int MT>
struct Up {
    static constexpr int kTok = 8, kRank = 16 * MT;
    static constexpr int kRow = (kRank + (MT == 1 ? 0 : 16)) * 2;  // bytes of a row of a term: four rows' reads lie in different banks
    static constexpr int kTerm = kTok * kRow, kU = (Terms<T>::n * kTerm + kTok * 4 + 1023) / 1024 * 1024;
    static constexpr int kBlocks = MT == 4 ? 2 : 3;
    // a warp's ring: a kilobyte of y (8 tokens, 32 outputs) and MT of B a stage
    static constexpr int kStage = 1024 + MT * 1024, kDepth = MT == 1 ? 3 : 2;
    static constexpr int kSmem = kU + kWarps * kDepth * kStage;
    static_assert(kSmem <= 228 * 1024 / kBlocks - 2048, "shared memory");
};

// y_out = y + B u over runs of 32 outputs: a block's warps take p.runs of them after another.
template <typename T, int MT>
__global__ void __launch_bounds__(kThreads, (Up<T, MT>::kBlocks)) lora_up_kernel(const __grid_constant__ LoraParams p) {
    using S = Up<T, MT>;
    constexpr int kTerms = Terms<T>::n;
    extern __shared__ __align__(16) uint8_t smem_up[];
    uint8_t *const u = smem_up;
    float *const back = reinterpret_cast<float *>(u + kTerms * S::kTerm);  // what takes a token's power of two out again
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3, mat = blockIdx.z;
    const float *y = p.d.y[mat];
    float *yo = p.d.y_out[mat];
    const int out = p.d.out[mat], groups = (out + 31) / 32, g0 = blockIdx.y * p.runs * kWarps + warp, g1 = min(groups, ((int)blockIdx.y + 1) * p.runs * kWarps);
    const Piece q = (int)blockIdx.y * p.runs * kWarps < groups ? find_piece<S::kTok>(p, blockIdx.x, y == yo, warp, lane, false) : Piece{};
    if (!q.n) {
        asm volatile("griddepcontrol.wait;\n" ::: "memory");  // every block: what follows this kernel also follows the one before it
        return;
    }
    const int64_t yo_st = p.d.y_out_stride[mat];
    int64_t y_st = p.d.y_stride[mat];
    const uint16_t *B = static_cast<const uint16_t *>(p.d.b[mat]) + (int64_t)max(q.adapter, 0) * out * p.d.rank;
    const bool vec_y = p.vec_y[mat], ring_b = p.vec_b;
    const int mine = g0 < g1 ? (g1 - g0 + kWarps - 1) / kWarps : 0;
    const uint32_t ring = smem_u32(smem_up) + S::kU + warp * S::kDepth * S::kStage;
    // Ranks in runs of kRank, each added to what the one before left (one run, nearly always).
#pragma unroll 1
    for (int r0 = 0; r0 == 0 || r0 < q.rank; r0 += S::kRank) {
        const int rank = min(S::kRank, q.rank - r0);
        // A lane's elements of its j-th run of outputs are copied some runs ahead of their turn.
        int sj = 0, sst = 0;
        auto send = [&]() {
            if (sj < mine) {
                const int o = (g0 + sj * kWarps) * 32 + 4 * g;
                const uint32_t to = ring + sst * S::kStage;
                if (vec_y) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int tok = 2 * c + h;
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
                ++sj;
            }
            copies_sent();
            if (++sst == S::kDepth) sst = 0;
        };
#pragma unroll 1
        for (int j = 0; j < S::kDepth - 1; ++j) send();
        if (r0) __syncthreads();  // u is read
        else asm volatile("griddepcontrol.wait;\n" ::: "memory");
        // ---------------------------------------------------------------- u in terms --
        if (rank > 0) {
            gather_u<T, S::kRank>(p, q, mat, r0, S::kTok, back, false, [&](int k, int t, int r, uint2 w) {
                *reinterpret_cast<uint2 *>(u + k * S::kTerm + t * S::kRow + r * 2) = w;
            });
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
            send();
            copies_landed<S::kDepth - 1>();
            const uint32_t at = ring + st * S::kStage;
            if (++st == S::kDepth) st = 0;
            if (ring_b) {
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int i = 0; i < 4; ++i) b[m][i] = lds8(at + 1024 + (m * 4 + i) * 256 + lane * 8);
                if (rank & 3) {  // (uniform) a run that ends inside four
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int i = 0; i < 4; ++i) b[m][i] = cut_b(b[m][i], rank - m * 16 - 4 * c);
                }
            }
            float v[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int tok = 2 * c + h;
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
            float d[2][2][4] = {};  // the first term's products, and the others'
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                if (m >= kts) break;
                const uint8_t *row = u + g * S::kRow + m * 32 + 8 * c;
#pragma unroll
                for (int k = kTerms - 1; k >= 0; --k) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(row + k * S::kTerm);
#pragma unroll
                    for (int f = 0; f < 2; ++f) mma16<T>(d[k > 0][f], b[m][2 * f].x, b[m][2 * f + 1].x, b[m][2 * f].y, b[m][2 * f + 1].y, w.x, w.y);
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int tok = 2 * c + h;
                if (tok >= q.n || n_o <= 0) continue;
                if (rank > 0) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float sum = d[0][i >> 1][2 * (i & 1) + h] + d[1][i >> 1][2 * (i & 1) + h];
                        v[h][i] = std::is_same<T, __half>::value ? fmaf(sum, back[tok], v[h][i]) : v[h][i] + sum;
                    }
                }
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
        copies_landed<0>();
        if (r0 + S::kRank < q.rank) __threadfence();  // copies will read what was stored
        y = yo, y_st = yo_st;
    }
}

// ------------------------------------------------------ many tokens: tcgen05 --
// The outputs are the M side (128 to a tile) and 64 tokens the N side, so that what a thread reads back from tensor memory is one output of
// 32 tokens: the lanes of a warp then meet y in whole lines, and an element costs a load, an addition and a store. The
// terms of u lie behind each other along K, the weights are used again for each.
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
// The issuing warp runs as a whole and one elected lane issues.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile(
        "{\n .reg .pred e;\n elect.sync _|e, 0xFFFFFFFF;\n"
        " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar)
        : "memory");
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p, e;\n elect.sync _|e, 0xFFFFFFFF;\n setp.ne.b32 p, %4, 0;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc));
}
// A K-major operand in 128-byte swizzled atoms of 8 rows of 128 bytes, atoms 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint32_t swizzled(int row, int byte) { return (uint32_t)((row >> 3) * 1024 + (row & 7) * 128 + (byte ^ ((row & 7) << 4))); }
__device__ __forceinline__ void tmem_ld16(uint32_t a, float (&v)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
                 "tcgen05.wait::ld.sync.aligned;\n"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
                   "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ bool poll(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity), "r"(1000u)
                 : "memory");
    return ok;
}
// A wait that is not over within p.spin polls marks the status word and sets `abort`, at which every wait of the block that is not over gives up (false).
// Who gave up sends no copy, product or arrival after it; what was sent is waited for at the block's end (drain).
__device__ __forceinline__ bool wait(const LoraParams &p, uint32_t bar, uint32_t parity, volatile int &abort) {
    for (unsigned i = 0; !poll(bar, parity); ++i) {
        if (abort) return false;
        if (i >= p.spin) {
            atomicOr(p.status, 0x474B0001u);
            abort = 1;
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool all(bool ok) { return __all_sync(0xFFFFFFFFu, ok); }
// The end of a copy or product that was sent, for a block that gave up.
__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity) {
    for (unsigned i = 0; i < kSpin && !poll(bar, parity); ++i) {}
}

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n" ::"r"(dst), "l"(map),
                 "r"(x), "r"(y), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) { asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory"); }
__device__ __forceinline__ void bar_sync(int id, int n) { asm volatile("barrier.cta.sync %0, %1;\n" ::"r"(id), "r"(n) : "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory"); }

template <typename T, int MT>
struct UpMany {
    static constexpr int kTok = 64, kOut = 128, kRank = 16 * MT, kSteps = MT * Terms<T>::n;  // of 16 along K
    static constexpr int kU = (kSteps + 3) / 4 * kTok * 128, kB = kOut * 128;  // 64 along K to a row of 128 bytes
    static constexpr int kYRow = kOut * 4, kY = kTok * kYRow;  // of y, a token's 128 outputs
    static constexpr int kStages = 2;
    static constexpr int oB = kU, oY = oB + kB, oBack = oY + kStages * kY, kSmem = oBack + kTok * 4 + 1024;  // (the atoms start on 1024 bytes)
    static constexpr int kBlocks = 2;
    static constexpr uint32_t kDesc = (1u << 4) | (std::is_same<T, __nv_bfloat16>::value ? 1u << 7 | 1u << 10 : 0u) | (uint32_t)(kTok >> 3) << 17 |
                                      (uint32_t)(kOut >> 4) << 24;
    static_assert(kSmem <= 228 * 1024 / kBlocks - 2048, "shared memory");
};
constexpr int kManyThreads = kThreads + 32;
// y and y_out as tensor maps: boxes of 128 outputs x 64 tokens.
struct UpMaps {
    CUtensorMap in[CQ_LORA_MAX_MATS], out[CQ_LORA_MAX_MATS];
};

// Eight warps compute: warp w has outputs 32 (w % 4) .. of a tile and tokens 32 (w / 4) .. of the piece. A ninth brings tiles of y by tensor
// copies and takes the results back from the same place. (BULK: rows start on 16 bytes. Else the eight read and write y themselves.) Ranks beyond kRank are summed in tensor memory, with u made anew for every tile.
template <typename T, int MT, bool BULK>
__global__ void __launch_bounds__(kManyThreads, (UpMany<T, MT>::kBlocks)) lora_up_many_kernel(const __grid_constant__ LoraParams p,
                                                                                               const __grid_constant__ UpMaps maps) {
    using S = UpMany<T, MT>;
    extern __shared__ uint8_t smem_many[];
    __shared__ uint64_t s_bars[2 + 2 * S::kStages];  // products done, y there, results there; one that nothing completes
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31, mat = blockIdx.z;
    const float *y = p.d.y[mat];
    float *yo = p.d.y_out[mat];
    const int out = p.d.out[mat], t0 = blockIdx.y * p.runs, tiles = min((out + S::kOut - 1) / S::kOut - t0, p.runs);  // of outputs
    const Piece q = tiles > 0 ? find_piece<S::kTok>(p, blockIdx.x, y == yo, warp, lane, false) : Piece{};
    if (!q.n) {
        asm volatile("griddepcontrol.wait;\n" ::: "memory");  // every block: what follows this kernel also follows the one before it
        return;
    }
    uint8_t *const smem = smem_many + (1024 - (smem_u32(smem_many) & 1023)) % 1024;
    float *const back = reinterpret_cast<float *>(smem + S::oBack);
    const uint32_t done = smem_u32(s_bars), full = done + 8, ready = full + 8 * S::kStages, base = smem_u32(smem);
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(&s_tmem)), "r"(S::kTok));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::);
    }
    if (tid == 0) {
        s_abort = 0;
        for (int i = 0; i < 2 + 2 * S::kStages; ++i)
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(done + 8 * i), "r"(i < 1 + S::kStages ? 1 : kWarps));
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const int64_t yo_st = p.d.y_out_stride[mat], y_st = p.d.y_stride[mat];
    // A tensor copy writes whole tiles: of a piece of fewer tokens each thread writes its own results. (A copy for each row instead held
    // the launch up: 8190 tokens of three requests 73 us against 64.)
    const bool whole = q.n == S::kTok;
    int sent = 0;  // tiles of y (the ninth warp's); products (the others')
    if (warp == kWarps) {
        if (BULK) {
            // A copy reads whole tiles, rows of the next piece among them.
            auto load = [&](int i) {
                sent = i + 1;
                if (lane == 0) {
                    const uint32_t bar = full + i % S::kStages * 8;
                    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(bar), "r"(S::kY) : "memory");
                    tma_load(base + S::oY + i % S::kStages * S::kY, &maps.in[mat], (t0 + i) * S::kOut, q.first, bar);
                }
            };
            for (int i = 0; i < S::kStages && i < tiles; ++i) load(i);
#pragma unroll 1
            for (int i = 0; i < tiles; ++i) {
                if (!all(wait(p, ready + i % S::kStages * 8, (uint32_t)(i / S::kStages) & 1, s_abort))) break;
                const uint32_t from = base + S::oY + i % S::kStages * S::kY;
                const int o = (t0 + i) * S::kOut;
                if (whole && lane == 0)
                    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];\n" ::"l"(&maps.out[mat]), "r"(o), "r"(q.first),
                                 "r"(from)
                                 : "memory");
                asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
                if (i + S::kStages < tiles) {
                    asm volatile("cp.async.bulk.wait_group.read 0;\n" ::: "memory");
                    __syncwarp();
                    load(i + S::kStages);
                }
            }
            asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory");
        }
        asm volatile("griddepcontrol.wait;\n" ::: "memory");
    } else {
        const uint16_t *B = static_cast<const uint16_t *>(p.d.b[mat]) + (int64_t)max(q.adapter, 0) * out * p.d.rank;
        const bool vec_b = p.d.rank % 8 == 0 && (reinterpret_cast<uintptr_t>(p.d.b[mat]) & 15) == 0;
        const int chunks = (q.rank + S::kRank - 1) / S::kRank;
        uint32_t par = 0;
        bool live = true;  // (of the issuing warp) products have come to their end so far
        // 128 rows of B, 8 ranks at a time, zeros where there is nothing
        auto fill = [&](int tile, int chunk) {
            const int r0 = chunk * S::kRank, rank = min(S::kRank, q.rank - r0);
#pragma unroll 1
            for (int i = tid; i < S::kOut * 2 * MT; i += kThreads) {
                const int row = i / (2 * MT), r = i % (2 * MT) * 8, o = (t0 + tile) * S::kOut + row, n = o < out ? rank - r : 0;
                const uint32_t to = base + S::oB + swizzled(row, r * 2);
                const uint16_t *from = B + (n > 0 ? (int64_t)o * p.d.rank + r0 + r : 0);
                if (n >= 8 && vec_b) {
                    copy16(to, from, true);
                } else {
                    const uint4 v = load_a(from, n);
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};\n" ::"r"(to), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
                }
            }
            copies_sent();
        };
        auto make_u = [&](int chunk) {
            gather_u<T, S::kRank>(p, q, mat, chunk * S::kRank, S::kTok, back, chunks > 1, [&](int k, int t, int r, uint2 w) {
                const int at = k * S::kRank + r;  // along K
                asm volatile("st.shared.v2.u32 [%0], {%1, %2};\n" ::"r"(base + (at >> 6) * (S::kTok * 128) + swizzled(t, (at & 63) * 2)), "r"(w.x), "r"(w.y)
                             : "memory");
            });
        };
        // What was filled is there, and all eight warps have read the products before.
        auto issue = [&](bool more) {
            copies_landed<0>();
            fence_async();
            fence_before();
            bar_sync(1, kThreads);
            if (warp || !live) return;
            ++sent;
            fence_after();
            const uint64_t a = desc_sw128(base + S::oB), b = desc_sw128(base);
            const uint32_t d = __shfl_sync(0xFFFFFFFFu, s_tmem, 0);
#pragma unroll
            for (int k = 0; k < S::kSteps; ++k) {  // the smallest terms first
                const int at = S::kSteps - MT + k % MT - k / MT * MT;
                mma_ss(d, a + (uint64_t)((k % MT) * 32 >> 4), b + (uint64_t)(((at >> 2) * (S::kTok * 128) + (at & 3) * 32) >> 4), S::kDesc, more || k);
            }
            mma_commit(done);
        };
        auto products = [&]() {
            const bool ended = wait(p, p.give_up ? done + 8 * (1 + 2 * S::kStages) : done, par, s_abort);
            if (warp == 0) live = all(live && ended);
            par ^= 1;
            fence_after();
        };
        // One power of two for all of a token's ranks, where they come in chunks.
        auto scale_all = [&]() {
            uint32_t *top = reinterpret_cast<uint32_t *>(back);
            for (int i = tid; i < S::kTok; i += kThreads) top[i] = 0;
            bar_sync(1, kThreads);
            const float *from = p.u + ((int64_t)mat * p.splits * p.d.n_tokens + q.first) * p.u_row;
            const int64_t next = (int64_t)p.d.n_tokens * p.u_row;
            for (int i = tid; i < q.n * chunks * S::kRank; i += kThreads) {
                const int t = i / (chunks * S::kRank), r = i - t * chunks * S::kRank;
                float x = 0.0f;
                for (int k = 0; k < p.splits; ++k) x += __ldcg(from + k * next + (int64_t)t * p.u_row + r);
                atomicMax(&top[t], magnitude(x));
            }
            bar_sync(1, kThreads);
            for (int i = tid; i < S::kTok; i += kThreads) back[i] = back_of(top[i]);
            bar_sync(1, kThreads);
        };
        // Every chunk of a tile whose ranks are many, but for the last one's wait.
        auto all_chunks = [&](int tile) {
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) {
                if (c) products();
                fill(tile, c);
                make_u(c);
                issue(c > 0);
            }
        };
        if (chunks == 1) fill(0, 0);
        asm volatile("griddepcontrol.wait;\n" ::: "memory");
        if (std::is_same<T, __half>::value && chunks > 1) scale_all();
        if (chunks == 1) make_u(0), issue(false);
        else all_chunks(0);
        const int tok0 = 32 * (warp >> 2), toks = min(32, q.n - tok0);
        const uint32_t from = base + S::oY + tok0 * S::kYRow + (32 * (warp & 3) + lane) * 4;
#pragma unroll 1
        for (int i = 0; i < tiles; ++i) {
            if (chunks) products();
            if (chunks == 1 && i + 1 < tiles) fill(i + 1, 0);
            const int o = (t0 + i) * S::kOut + 32 * (warp & 3) + lane;
            const uint32_t mine = from + i % S::kStages * S::kY;
            bool there = true;
            if (BULK) there = wait(p, full + i % S::kStages * 8, (uint32_t)(i / S::kStages) & 1, s_abort);
            const float *src = y + (int64_t)(q.first + min(tok0, q.n - 1)) * y_st + min(o, out - 1);  // (what is not there: the last one again)
            float *dst = yo + (int64_t)(q.first + tok0) * yo_st + o;
#pragma unroll
            for (int h = 0; h < 32; h += 16) {
                if (BULK && whole && !chunks) continue;  // y goes back as it came
                float d[16] = {}, v[16];
                if (chunks) tmem_ld16(s_tmem + ((uint32_t)(32 * (warp & 3)) << 16) + tok0 + h, d);
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    if (BULK) {
                        asm volatile("ld.shared.f32 %0, [%1];\n" : "=f"(v[k]) : "r"(mine + (h + k) * S::kYRow));
                    } else {
                        asm volatile("ld.global.cs.f32 %0, [%1];\n" : "=f"(v[k]) : "l"(src));
                        if (h + k + 1 < toks) src += y_st;
                    }
                }
#pragma unroll
                for (int k = 0; k < 16; k += 4) {
                    if (!chunks) continue;
                    if (std::is_same<T, __half>::value) {
                        const float4 f = *reinterpret_cast<const float4 *>(back + tok0 + h + k);
                        v[k] = fmaf(d[k], f.x, v[k]), v[k + 1] = fmaf(d[k + 1], f.y, v[k + 1]);
                        v[k + 2] = fmaf(d[k + 2], f.z, v[k + 2]), v[k + 3] = fmaf(d[k + 3], f.w, v[k + 3]);
                    } else {
                        v[k] += d[k], v[k + 1] += d[k + 1], v[k + 2] += d[k + 2], v[k + 3] += d[k + 3];
                    }
                }
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    if (BULK && whole) {
                        asm volatile("st.shared.f32 [%0], %1;\n" ::"r"(mine + (h + k) * S::kYRow), "f"(v[k]) : "memory");
                    } else {
                        if (h + k < toks && o < out) *dst = v[k];
                        dst += yo_st;
                    }
                }
            }
            if (BULK) {
                fence_async();
                __syncwarp();
                if (lane == 0 && there) mbar_arrive(ready + i % S::kStages * 8);
            }
            if (i + 1 < tiles) {
                if (chunks == 1) issue(false);
                else if (chunks) all_chunks(i + 1);
            }
        }
        fence_before();
    }
    __syncthreads();
    if (s_abort) {  // no wait of a block that gave up says that these have ended
        if (warp == kWarps)
            for (int i = max(0, sent - S::kStages); i < sent; ++i) drain(full + i % S::kStages * 8, (uint32_t)(i / S::kStages) & 1);
        else if (warp == 0 && sent) drain(done, (uint32_t)(sent - 1) & 1);
        __syncwarp();
    }
    if (warp == 0) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(s_tmem), "r"(S::kTok));
    }
}

// The first product on tcgen05: 128 tokens are the M side, the ranks the N side, 64 inputs a stage. One warp brings stages by tensor copies, one
// issues; four read the sums back, and turn int8 stages into the weights' type before that.
struct DownMaps {
    CUtensorMap x, a[CQ_LORA_MAX_MATS];
};
template <typename T, int XK, int MT>
struct DownMany {
    static constexpr int kTok = 128, kRank = 16 * MT, kIn = 64;
    static constexpr int kX = kTok * 128, kA = kRank * 128, kRaw = XK == CQ_T_I8 ? kTok * 64 : 0, kStage = kX + kA + kRaw;
    static constexpr int kBlocks = 2, kRoom = 228 * 1024 / kBlocks - 2048 - 1024;  // (stages start on 1024 bytes)
    static constexpr int kDepth = kRoom / kStage < 6 ? kRoom / kStage : 6, kSmem = kDepth * kStage + 1024;
    static constexpr int kCols = kRank < 32 ? 32 : kRank;
    static constexpr uint32_t kDesc = (1u << 4) | (std::is_same<T, __nv_bfloat16>::value ? 1u << 7 | 1u << 10 : 0u) | (uint32_t)(kRank >> 3) << 17 |
                                      (uint32_t)(kTok >> 4) << 24;
    static_assert(kDepth >= 2, "shared memory");
};
constexpr int kDownThreads = 192;

template <typename T, int XK, int MT>
__global__ void __launch_bounds__(kDownThreads, (DownMany<T, XK, MT>::kBlocks)) lora_down_many_kernel(const __grid_constant__ LoraParams p,
                                                                                                     const __grid_constant__ DownMaps maps) {
    using S = DownMany<T, XK, MT>;
    extern __shared__ uint8_t smem_down[];
    __shared__ uint64_t s_bars[3 * S::kDepth + 2];  // stages there, turned, free; the sums done; one that nothing completes
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
    const int cut = blockIdx.x % p.splits, mat = blockIdx.y, r0 = blockIdx.z * S::kRank;
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const Piece q = find_piece<S::kTok>(p, blockIdx.x / p.splits, true, warp, lane, blockIdx.x + blockIdx.y + blockIdx.z == 0);
    const int rank = min(S::kRank, q.rank - r0);
    if (!q.n || rank <= 0) return;
    const int chunks = (p.d.in + S::kIn - 1) / S::kIn, c0 = (int)((long long)chunks * cut / p.splits), n = (int)((long long)chunks * (cut + 1) / p.splits) - c0;
    const uint32_t base = (smem_u32(smem_down) + 1023) & ~1023u, full = smem_u32(s_bars), turned = full + 8 * S::kDepth, empty = turned + 8 * S::kDepth,
                   done = empty + 8 * S::kDepth;
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(&s_tmem)), "r"(S::kCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::);
    }
    if (tid == 0) {
        s_abort = 0;
        for (int i = 0; i < 3 * S::kDepth + 2; ++i)
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(full + 8 * i), "r"(i >= S::kDepth && i < 2 * S::kDepth ? 4 : 1));
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    int sent = 0;  // stages (lane 0 of warp 0)
    if (warp == 0) {
        if (lane == 0) {
#pragma unroll 1
            for (int i = 0; i < n; ++i) {
                const int st = i % S::kDepth;
                const uint32_t at = base + st * S::kStage, bar = full + 8 * st;
                if (i >= S::kDepth && !wait(p, empty + 8 * st, (uint32_t)(i / S::kDepth - 1) & 1, s_abort)) break;
                sent = i + 1;
                asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(bar), "r"((XK == CQ_T_I8 ? S::kRaw : S::kX) + S::kA) : "memory");
                tma_load(XK == CQ_T_I8 ? at + S::kX + S::kA : at, &maps.x, (c0 + i) * S::kIn, q.first, bar);
                tma_load(at + S::kX, &maps.a[mat], (c0 + i) * S::kIn, q.adapter * p.d.rank + r0, bar);
            }
        }
    } else if (warp == 1) {
        const uint32_t d = __shfl_sync(0xFFFFFFFFu, s_tmem, 0);
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            const int st = i % S::kDepth;
            const uint32_t par = (uint32_t)(i / S::kDepth) & 1;
            bool there = wait(p, p.give_up ? done + 8 : full + 8 * st, par, s_abort);
            if (XK == CQ_T_I8) there = wait(p, turned + 8 * st, par, s_abort) && there;
            if (!all(there)) break;
            fence_after();
            const uint64_t a = desc_sw128(base + st * S::kStage), b = desc_sw128(base + st * S::kStage + S::kX);
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_ss(d, a + (uint64_t)(k * 32 >> 4), b + (uint64_t)(k * 32 >> 4), S::kDesc, (i | k) != 0);
            mma_commit(empty + 8 * st);
        }
        mma_commit(done);
    } else {
        const int row = 32 * (warp & 3) + lane;
        if (XK == CQ_T_I8) {
#pragma unroll 1
            for (int i = 0; i < n; ++i) {  // a token to a thread
                const int st = i % S::kDepth;
                const uint32_t to = base + st * S::kStage, from = to + S::kX + S::kA + row * 64;
                if (!all(wait(p, full + 8 * st, (uint32_t)(i / S::kDepth) & 1, s_abort))) break;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint4 v = lds16(from + ((j ^ (row >> 1 & 3)) << 4));  // 16 inputs, 64-byte swizzled
                    uint32_t w[4];
                    const uint32_t lo[2] = {v.x, v.y}, hi[2] = {v.z, v.w};
                    pairs_of_i8<T>(lo, w);
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};\n" ::"r"(to + swizzled(row, 32 * j)), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                                 : "memory");
                    pairs_of_i8<T>(hi, w);
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};\n" ::"r"(to + swizzled(row, 32 * j + 16)), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                                 "r"(w[3])
                                 : "memory");
                }
                fence_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(turned + 8 * st);
            }
        }
        float scale = p.d.scales ? p.d.scales[q.adapter] : 1.0f, own = 1.0f;
        if (XK == CQ_T_I8) own = p.d.x_scale[q.first + min(row, q.n - 1)];
        wait(p, done, 0, s_abort);
        fence_after();
        float *u = p.u + (((int64_t)mat * p.splits + cut) * p.d.n_tokens + q.first + row) * p.u_row + r0;
#pragma unroll
        for (int h = 0; h < S::kRank; h += 16) {
            float v[16];
            tmem_ld16(s_tmem + ((uint32_t)(32 * (warp & 3)) << 16) + h, v);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                if (XK == CQ_T_I8) v[j] *= own;
                v[j] = h + j < rank ? v[j] * scale : 0.0f;  // ranks that are not there hold what other rows gave
            }
            if (row < q.n) {
#pragma unroll
                for (int j = 0; j < 16; j += 4) *reinterpret_cast<float4 *>(u + h + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
            }
        }
        fence_before();
    }
    __syncthreads();
    if (s_abort) {  // no wait of a block that gave up says that these have ended
        for (int i = max(0, sent - S::kDepth); i < sent; ++i) drain(full + 8 * (i % S::kDepth), (uint32_t)(i / S::kDepth) & 1);
        if (warp == 1) drain(done, 0);
        __syncwarp();
    }
    if (warp == 1) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(s_tmem), "r"(S::kCols));
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
// A tensor map over rows of `width` elements: boxes of box_x x box_y.
inline int make_map(CUtensorMap *map, CUtensorMapDataType type, int size, const void *at, int width, long long rows, int64_t stride, int box_x, int box_y,
                    CUtensorMapSwizzle swizzle) {
    typedef CUresult (*Encode)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                               const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static Encode fn = nullptr;  // every writer stores the same value
    if (!fn) {
        cudaDriverEntryPointQueryResult found;
        void *f = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess || !f) {
            cudaGetLastError();
            return set_error(CQ_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
        }
        fn = reinterpret_cast<Encode>(f);
    }
    if (rows == 1) stride = (int64_t)(width + 15) / 16 * 16;  // of no meaning, but checked
    const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)stride * size};
    const cuuint32_t box[2] = {(cuuint32_t)box_x, (cuuint32_t)box_y}, one[2] = {1, 1};
    const CUresult r = fn(map, type, 2, const_cast<void *>(at), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? CQ_OK : set_error(CQ_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
}
template <typename T, int XK, int MT>
int launch_down_many(const LoraParams &p, cudaStream_t st) {
    using S = DownMany<T, XK, MT>;
    auto k = lora_down_many_kernel<T, XK, MT>;
    const CUtensorMapDataType type = std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    DownMaps maps;
    int rc = XK == CQ_T_I8 ? make_map(&maps.x, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, p.d.x, p.d.in, p.d.n_tokens, p.d.x_stride, S::kIn, S::kTok, CU_TENSOR_MAP_SWIZZLE_64B)
                           : make_map(&maps.x, type, 2, p.d.x, p.d.in, p.d.n_tokens, p.d.x_stride, S::kIn, S::kTok, CU_TENSOR_MAP_SWIZZLE_128B);
    for (int j = 0; !rc && j < p.d.n_mats; ++j)
        rc = make_map(&maps.a[j], type, 2, p.d.a[j], p.d.in, (long long)p.d.n_adapters * p.d.rank, p.d.in, S::kIn, S::kRank, CU_TENSOR_MAP_SWIZZLE_128B);
    if (!rc) rc = ensure_smem(reinterpret_cast<const void *>(k), S::kSmem);
    if (rc) return rc;
    k<<<dim3(p.pieces * p.splits, p.d.n_mats, p.u_row / S::kRank), kDownThreads, S::kSmem, st>>>(p, maps);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? CQ_OK : set_error(CQ_ERR_CUDA, "adapter launch: %s", cudaGetErrorString(e));
}

// The kernel of the second product behind the first's: begun before that one has ended.
template <typename K, typename... A>
int launch_after(K k, dim3 grid, int threads, int smem, cudaStream_t st, const A &...args) {
    if (smem > 48 * 1024) {
        const int rc = ensure_smem(reinterpret_cast<const void *>(k), smem);
        if (rc) return rc;
    }
    if (grid.y > 65535) return set_error(CQ_ERR_SHAPE, "too many outputs for one call");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, k, args...);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e == cudaSuccess) return CQ_OK;
    cudaGetLastError();
    return set_error(CQ_ERR_CUDA, "adapter launch: %s", cudaGetErrorString(e));
}
template <typename T, int MT>
int launch_up(LoraParams &p, cudaStream_t st) {
    const int tile = p.few ? 32 * kWarps : UpMany<T, MT>::kOut;
    const long long pieces = p.few ? p.pieces : std::min<long long>(p.d.n_tokens, (long long)p.d.n_seqs + p.d.n_tokens / UpMany<T, MT>::kTok);
    const long long room = (long long)sm_count() * (p.few ? Up<T, MT>::kBlocks : UpMany<T, MT>::kBlocks);
    int tiles = 1;  // of the widest matrix
    for (int j = 0; j < p.d.n_mats; ++j) tiles = std::max(tiles, (p.d.out[j] + tile - 1) / tile);
    // Tiles that a block takes after another: a block's beginning costs about as much as two, and blocks that do not fit wait for others.
    long long best = LLONG_MAX;
    p.runs = 1;
    for (int parts = 1; parts <= tiles; parts += parts < 16 ? 1 : parts) {
        const int r = (tiles + parts - 1) / parts;
        long long blocks = 0;
        for (int j = 0; j < p.d.n_mats; ++j) blocks += pieces * (((p.d.out[j] + tile - 1) / tile + r - 1) / r);
        const long long cost = (blocks + room - 1) / room * (r + 2);
        if (cost < best) best = cost, p.runs = r;
    }
    const dim3 grid((unsigned)pieces, (unsigned)((tiles + p.runs - 1) / p.runs), (unsigned)p.d.n_mats);
    if (p.few) return launch_after(lora_up_kernel<T, MT>, grid, kThreads, Up<T, MT>::kSmem, st, p);
    using S = UpMany<T, MT>;
    UpMaps maps;
    bool bulk = true;
    for (int j = 0; j < p.d.n_mats; ++j) bulk = bulk && p.vec_y[j];
    if (!bulk) return launch_after(lora_up_many_kernel<T, MT, false>, grid, kManyThreads, S::kSmem, st, p, maps);
    for (int j = 0; j < p.d.n_mats; ++j) {
        int rc = make_map(&maps.in[j], CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, p.d.y[j], p.d.out[j], p.d.n_tokens, p.d.y_stride[j], S::kOut, S::kTok,
                          CU_TENSOR_MAP_SWIZZLE_NONE);
        if (!rc) rc = make_map(&maps.out[j], CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, p.d.y_out[j], p.d.out[j], p.d.n_tokens, p.d.y_out_stride[j], S::kOut, S::kTok,
                               CU_TENSOR_MAP_SWIZZLE_NONE);
        if (rc) return rc;
    }
    return launch_after(lora_up_many_kernel<T, MT, true>, grid, kManyThreads, S::kSmem, st, p, maps);
}

template <typename T, int XK, int MT, bool VEC>
int launch_r(LoraParams &p, cudaStream_t st) {
    constexpr int WT = lora_warps_along(false), NT = lora_tokens(XK, MT, false, false) / (8 * WT);
    int rc;
    if (VEC && p.few) rc = launch_down<T, XK, MT, 1, 1, true>(p, st);
    else if (VEC && XK != CQ_T_F32 && p.tensor) rc = launch_down_many<T, XK == CQ_T_F32 ? CQ_T_F16 : XK, MT>(p, st);
    else rc = launch_down<T, XK, MT, NT, WT, VEC>(p, st);
    if (rc) return rc;
    return launch_up<T, MT>(p, st);
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
    p.spin = p.give_up ? 4 : kSpin;
    if (p.d.x_dtype == CQ_T_F32) return p.vec ? launch_x<T, CQ_T_F32, true>(p, st) : launch_x<T, CQ_T_F32, false>(p, st);
    if (p.d.x_dtype == CQ_T_I8) return p.vec ? launch_x<T, CQ_T_I8, true>(p, st) : launch_x<T, CQ_T_I8, false>(p, st);
    return p.vec ? launch_x<T, CQ_T_F16, true>(p, st) : launch_x<T, CQ_T_F16, false>(p, st);
}

}  // namespace
}  // namespace cq
