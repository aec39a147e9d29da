// cq_tree.cu -- attention of drafted tokens over a paged CQ cache, on tcgen05.
//
// Mathematics. With the rotated-domain identity a logit is
//   x[c][t] = scale * n_k[t] * <levels(codes_k[t]), z[c]>,  z[c] = H q[c],
// c a column (a drafted token and one of its query heads), t a cache row, and
//   o[c] = H sum_t p[c][t] n_v[t] levels(codes_v[t]) / sum_t p[c][t],
// so neither cache is rotated back: two matrix products run on bare level tables and one rotation
// per column ends the work. The query heads of a unit (see TreeUnit) share the codes of its groups:
// a drafted token makes `rows` columns, and a tile of 128 cache rows is expanded once for N columns.
//
// Layout. Cache rows are the M side of the first product (S^T[128 rows][N] = K Z^T) and the value
// coordinates the M side of the second (O^T[128][N] += V^T P^T): N is the number of columns, 16 for
// one token and 128 for a large tree, and no tensor work is spent on columns that are not there. A
// softmax thread owns a cache row, so that row's norms are registers, not loads.
//
// Exponents. The norm of a value row goes into the exponent:
//   w[c][t] = 2^(x log2(e) + log2 n_v[t] - m[c]),  o = H sum_t w levels / sum_t w / n_v[t].
// w is what the second product takes in fp16 (one rounding of 2^-11); with the reference m from the
// column's own largest w it neither over- nor underflows whatever the size of the norms. m rises only when a
// column's w would pass 2^8 (the accumulators are then scaled, which is rare after the first tile); columns
// decide for themselves, so a column's bits do not depend on the others.
//
// Split. The tiles of all (request, unit, column tile) items in one row are cut into equal runs, one per SM:
// lengths are read on the device, and the longest request cannot hold the launch up. Each run leaves
// unrotated partial sums; a second kernel joins them, rotates and writes o.
//
// Roles of the 16 warps: 0-7 softmax (two warpgroups, half the columns each; they also rotate the queries
// and write the partials), 8-11 expand keys into TMEM (a thread per cache row; the A operand), 12-15
// expand values into shared memory; warp 8 also issues the first product of each tile and warp 12 the second. The expanders fetch their own codes by cp.async into a
// ring a few tiles ahead, so they wait for nobody's loads but their own. (A warp of its own for the MMAs would
// cost every thread a fifth of its registers: they are handed out to four warps at a time.)
// Every wait is bounded: when one gives up, the flag s_abort makes all later waits return at once and every role
// runs through its remaining tiles without waiting, so that the block's barriers stay matched.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>

#include "cq_paged.h"

namespace cq {
namespace {

constexpr int kTile = 128;        // cache rows per tile
constexpr int kSoftThreads = 256;
constexpr int kThreads = 512;
constexpr unsigned kSpin = 1u << 20;   // polls of up to ~1 us
constexpr float kNoMax = -1e30f;       // reference of a column that has attended nothing yet
constexpr float kRaise = 8.0f;         // log2 of the largest weight before a reference is raised
constexpr float kInvSqrt128 = 0.08838834764831845f;

struct TreeParams {
    cq_kv_tree t;
    TreeUnit unit[kMaxUnits];
    unsigned int *status;
    float *part;     // [slot][group][N][128] partial sums, unrotated
    float2 *ml;      // [slot][N] reference and denominator
    int2 *rec;       // [item] first slot and number of parts
    uint32_t tk[8], tv[8];  // level tables: low bytes of 16 fp16 levels, then high bytes
    float k_mult, v_mult;   // scale * log2(e) / sqrt(128) * 2^(table exponent); 2^(table exponent) / sqrt(128)
    int n_units, hq, per, dk, dv, wk, wv, kgroups, vgroups;
    uint32_t div_mul, div_shift;  // t / block_size = t * div_mul >> div_shift
    int rows;        // most query heads of a unit
    int ncol_max;    // column tiles of a request with max_nodes tokens
    int grid;
};

// ----------------------------------------------------------------------- PTX --
__device__ __forceinline__ uint32_t smem_u32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void mbar_init(uint64_t *bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(smem_u32(bar)), "r"(count));
}
__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(ok)
                 : "r"(smem_u32(bar)), "r"(parity)
                 : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool mbar_try(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(ok)
                 : "r"(smem_u32(bar)), "r"(parity), "r"(1000u)
                 : "memory");
    return ok != 0;
}
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }
// The issuing warp runs as a whole and one elected lane issues: operands then stay in uniform registers (a branch
// to one lane made each MMA cost about 100 cycles of moves).
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
    asm volatile(
        "{\n .reg .pred e;\n elect.sync _|e, 0xFFFFFFFF;\n"
        " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar))
        : "memory");
}
// D += A B with A in tensor memory (lane = row, a column holds two fp16) or in shared memory.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p, e;\n elect.sync _|e, 0xFFFFFFFF;\n setp.ne.b32 p, %4, 0;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p, e;\n elect.sync _|e, 0xFFFFFFFF;\n setp.ne.b32 p, %4, 0;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc));
}
// Shared-memory operand in 128-byte swizzled atoms of 8 rows of 128 bytes, atoms 1024 bytes apart
// along the rows. K-major: a row is one M/N index, 64 of K. MN-major: a row is one K index, 64 of M/N,
// and the next 64 of M/N lie `seg` bytes on.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr, uint32_t seg) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((seg >> 4) & 0x3FFFu) << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) |
           (2ull << 61);
}
// kind::f16, fp16 operands, fp32 accumulator; the last two: operand is MN-major.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int a_mn, int b_mn) {
    return (1u << 4) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
template <int X> __device__ __forceinline__ void tmem_ld(uint32_t a, float *v);
template <> __device__ __forceinline__ void tmem_ld<8>(uint32_t a, float *v) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "r"(a));
}
template <> __device__ __forceinline__ void tmem_ld<16>(uint32_t a, float *v) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
                   "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
                 : "r"(a));
}
template <> __device__ __forceinline__ void tmem_ld<32>(uint32_t a, float *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,"
        "%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]),
          "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]),
          "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]),
          "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(a));
}
// Waits for the loads into v; nothing that uses v moves above it.
template <int X> __device__ __forceinline__ void wait_ld(float *v) {
    asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
#pragma unroll
    for (int i = 0; i < X; ++i) asm volatile("" : "+f"(v[i]));
}
__device__ __forceinline__ void tmem_st8(uint32_t a, const float *v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(a), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                 "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t *v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(a),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
                 "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
                 : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];\n" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};\n" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t v) { asm volatile("st.shared.u32 [%0], %1;\n" ::"r"(a), "r"(v) : "memory"); }
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory"); }
__device__ __forceinline__ void bar_sync(int id, int n) { asm volatile("barrier.cta.sync %0, %1;\n" ::"r"(id), "r"(n) : "memory"); }
__device__ __forceinline__ bool bar_or(int id, int n, bool v) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"((uint32_t)v), "r"(id), "r"(n)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t s) { return __byte_perm(a, b, s); }

// ------------------------------------------------------------------ schedule --
// One request as the kernel takes it: lengths outside the given sizes are cut to
// them (`bad`), so that no index leaves its buffer whatever the device holds.
struct Seq {
    int first, n, ctx, len;
    bool bad;
};
__device__ __forceinline__ Seq seq_at(const TreeParams &p, int s) {
    Seq q;
    const int a = p.t.cu_nodes[s], b = p.t.cu_nodes[s + 1];
    long long ctx = p.t.context_lens[s];
    q.first = a;
    q.bad = a < 0 || b < a || b > p.t.n_nodes;
    q.n = q.bad ? 0 : min(b - a, p.t.max_nodes);
    q.bad |= !q.bad && b - a > p.t.max_nodes;
    const long long room = min((long long)p.t.max_blocks * p.t.block_size, (long long)INT_MAX);
    if (ctx < 0) q.bad = true, ctx = 0;
    q.bad |= q.n && ctx + q.n > room;
    q.ctx = (int)ctx;
    q.len = q.n ? (int)min(ctx + q.n, room) : 0;
    return q;
}
__device__ __forceinline__ int tiles_of(int len) { return max(1, (int)(((long long)len + kTile - 1) / kTile)); }
__device__ __forceinline__ int cols_of(const TreeParams &p, int n, int N) { return (n * p.rows + N - 1) / N; }

// A position in the row of all tiles.
struct Cursor {
    int s, u, c, tile, ntiles, ncol, first, n, ctx, len;
    int item;        // items before this one
    long long left;  // tiles of this block's run from here on
    __device__ void take(const TreeParams &p, int N) {
        const Seq q = seq_at(p, s);
        first = q.first, n = q.n, ctx = q.ctx, len = q.len;
        ntiles = tiles_of(len);
        ncol = cols_of(p, n, N);
    }
    __device__ void next_item(const TreeParams &p, int N) {
        tile = 0;
        ++item;
        if (++c < ncol) return;
        c = 0;
        if (++u < p.n_units) return;
        u = 0;
        do {
            if (++s >= p.t.n_seqs) return;
            take(p, N);
        } while (!n);
    }
    __device__ bool advance(const TreeParams &p, int N) {  // to the next tile; false after the last
        if (--left <= 0) return false;
        if (++tile == ntiles) next_item(p, N);
        return true;
    }
};

// Run b of `grid` blocks; with fewer tiles than blocks the first `total` blocks take one each, so that the parts of an
// item are consecutive blocks.
__device__ __forceinline__ long long run_start(long long total, int grid, int b) {
    const long long n = min(total, (long long)grid);
    return b < n ? total * b / n : total;
}
__device__ __forceinline__ int run_of(long long total, int grid, long long tile) {
    return (int)(((tile + 1) * min(total, (long long)grid) - 1) / total);
}

struct Shared {
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], s_empty[2], p_full[2], p_empty[2], sc_full[2], z_full, drain[2];
    uint32_t tmem;
    volatile int abort;
    int zmax;
    int bad;
    long long total, w0;          // all tiles; this block's first one
    long long scan_t[kThreads / 32];
    long long scan_i[kThreads / 32];
    Cursor start;
    float scal[2][3][kTile];      // per tile buffer: n_k, log2 n_v, 1 / n_v
    alignas(16) float m[128];     // column references (read four at a time)
    float f[128];                 // factors of the last raise
    float wmax[8][64];            // column maxima of a softmax warp
    float lsum[8][64];
    uint32_t mask[CQ_TREE_MAX_NODES][4];  // columns (bits) that attend drafted token j
};

__device__ __forceinline__ void wait(Shared &sh, uint64_t *bar, uint32_t parity, unsigned int *status, unsigned code) {
    if (mbar_test(bar, parity)) return;
    for (unsigned i = 0; !sh.abort; ++i) {
        if (mbar_try(bar, parity)) return;
        if (i >= kSpin) {
            atomicOr(status, code);
            sh.abort = 1;
        }
    }
}

// Fills sh.start with this block's first tile and sh.total; false if it has none.
template <int N>
__device__ bool find_run(const TreeParams &p, Shared &sh) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kW = kThreads / 32;
    auto tiles_and_items = [&](int s, long long &t, long long &i) {
        const Seq q = seq_at(p, s);
        if (q.bad) sh.bad = 1;
        i = (long long)p.n_units * cols_of(p, q.n, N);
        t = q.n ? i * tiles_of(q.len) : 0;
    };
    long long t = 0;
    for (int s = tid; s < p.t.n_seqs; s += kThreads) {
        long long a, b;
        tiles_and_items(s, a, b);
        t += a;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
    if (lane == 0) sh.scan_t[warp] = t;
    __syncthreads();
    long long total = 0;
    for (int w = 0; w < kW; ++w) total += sh.scan_t[w];
    __syncthreads();
    const long long w0 = run_start(total, p.grid, blockIdx.x), w1 = run_start(total, p.grid, blockIdx.x + 1);
    if (tid == 0) sh.total = total, sh.w0 = w0;
    if (w0 >= w1) return false;
    long long ct = 0, ci = 0;  // tiles and items before the chunk
    for (int base = 0; base < p.t.n_seqs; base += kThreads) {
        long long a = 0, b = 0;
        if (base + tid < p.t.n_seqs) tiles_and_items(base + tid, a, b);
        long long ia = a, ib = b;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long ua = __shfl_up_sync(0xFFFFFFFFu, ia, o), ub = __shfl_up_sync(0xFFFFFFFFu, ib, o);
            if (lane >= o) ia += ua, ib += ub;
        }
        if (lane == 31) sh.scan_t[warp] = ia, sh.scan_i[warp] = ib;
        __syncthreads();
        long long ba = ct, bb = ci;
        for (int w = 0; w < kW; ++w) {
            if (w < warp) ba += sh.scan_t[w], bb += sh.scan_i[w];
            ct += sh.scan_t[w], ci += sh.scan_i[w];
        }
        const long long t0 = ba + ia - a;
        if (a && t0 <= w0 && w0 < t0 + a) {  // exactly one thread
            Cursor c;
            c.s = base + tid;
            c.take(p, N);
            const long long off = w0 - t0;
            const int it = (int)(off / c.ntiles);
            c.tile = (int)(off - (long long)it * c.ntiles);
            c.u = it / c.ncol;
            c.c = it - c.u * c.ncol;
            c.item = (int)(bb + ib - b) + it;
            c.left = w1 - w0;
            sh.start = c;
        }
        __syncthreads();
        if (ct > w0) break;  // uniform
    }
    return true;
}

// --------------------------------------------------------------------- codes --
// Expanding codes. A byte permute looks four codes up at once in eight table bytes, so the low and the high
// bytes of four levels are two permutes, and two more interleave them into fp16 pairs: no memory access and 1.3
// (2 bits) to 2.5 (4 bits) instructions per value. Two-bit codes come out in the order 0, 2, .. 14, 1, 3,
// .. 15 of each 16 (position_of); the queries are stored in that order and the partial sums put back.
__device__ __forceinline__ int position_of(int k, int w) { return w == 2 ? (k & ~15) | (k & 1) << 3 | (k & 15) >> 1 : k; }
__device__ __forceinline__ int natural_of(int pos, int w) { return w == 2 ? (pos & ~15) | (pos & 7) << 1 | (pos & 15) >> 3 : pos; }

__device__ __forceinline__ void pairs_of(uint32_t lo, uint32_t hi, uint32_t *r) {
    r[0] = prmt(lo, hi, 0x5140);
    r[1] = prmt(lo, hi, 0x7362);
}
__device__ __forceinline__ void expand_w2(uint32_t x, const uint32_t (&t)[8], uint32_t *r) {  // 16 codes
    const uint32_t e = x & 0x33333333u, o = (x >> 2) & 0x33333333u;
    pairs_of(prmt(t[0], 0, e), prmt(t[4], 0, e), r);
    pairs_of(prmt(t[0], 0, e >> 16), prmt(t[4], 0, e >> 16), r + 2);
    pairs_of(prmt(t[0], 0, o), prmt(t[4], 0, o), r + 4);
    pairs_of(prmt(t[0], 0, o >> 16), prmt(t[4], 0, o >> 16), r + 6);
}
__device__ __forceinline__ void expand_w3(uint32_t x, const uint32_t (&t)[8], uint32_t *r) {  // 8 codes in the low 24 bits
    x = (x & 0x00000FFFu) | (x & 0x00FFF000u) << 4;
    x = (x & 0x003F003Fu) | (x & 0x0FC00FC0u) << 2;
    x = (x & 0x07070707u) | (x & 0x38383838u) << 1;
    pairs_of(prmt(t[0], t[1], x), prmt(t[4], t[5], x), r);
    pairs_of(prmt(t[0], t[1], x >> 16), prmt(t[4], t[5], x >> 16), r + 2);
}
__device__ __forceinline__ void expand_w4(uint32_t x, const uint32_t (&t)[8], uint32_t *r) {  // 8 codes
    const uint32_t s = x & 0x77777777u, h = (x >> 3) & 0x11111111u;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t si = s >> (16 * i), m = prmt(0x0000FF00u, 0, h >> (16 * i));  // 0xFF where the code is 8 or more
        const uint32_t lo = (prmt(t[0], t[1], si) & ~m) | (prmt(t[2], t[3], si) & m);
        const uint32_t hi = (prmt(t[4], t[5], si) & ~m) | (prmt(t[6], t[7], si) & m);
        pairs_of(lo, hi, r + 2 * i);
    }
}
// 32 codes, the q-th quarter of a group held in words c, as 16 fp16 pairs.
template <int W>
__device__ __forceinline__ void expand_quarter(const uint32_t *c, const uint32_t (&t)[8], uint32_t (&r)[16]) {
    if (W == 2) {
        expand_w2(c[0], t, r);
        expand_w2(c[1], t, r + 8);
    } else if (W == 3) {
        expand_w3(c[0] & 0xFFFFFFu, t, r);
        expand_w3(__funnelshift_r(c[0], c[1], 24) & 0xFFFFFFu, t, r + 4);
        expand_w3(__funnelshift_r(c[1], c[2], 16) & 0xFFFFFFu, t, r + 8);
        expand_w3(c[2] >> 8, t, r + 12);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) expand_w4(c[i], t, r + 4 * i);
    }
}

// ---------------------------------------------------------------- the kernel --
template <int N, int NG>
struct Plan {
    static constexpr int kVBuf = NG == 1 ? 2 : 1;
    static constexpr int kDepth = NG == 2 ? 2 : N >= 128 ? 3 : N >= 64 ? 4 : 6;  // tiles of codes in flight
    static constexpr int kVBytes = 2 * kTile * 128;            // one group's values: 128 rows x 128 fp16
    static constexpr int kPBytes = kTile * (N <= 64 ? 128 : 256);
    static constexpr int kZBytes = N * 256;                    // one group
    static constexpr int kRing = NG * 4 * kTile * 16;          // one stage of one side (four-bit codes)
    static constexpr int kNorm = NG * kTile * 4;
    static constexpr int oV = 0, oP = oV + kVBuf * NG * kVBytes, oZ = oP + 2 * kPBytes, oRing = oZ + NG * kZBytes;
    static constexpr int oNorm = oRing + 2 * kDepth * kRing, oShared = oNorm + 2 * kDepth * kNorm;
    static constexpr int kSmem = oShared + (int)sizeof(Shared) + 1024;
    static constexpr int kSoft = NG == 2 ? 136 : 160, kExp = 256 - kSoft;  // registers of the roles
    // TMEM columns
    static constexpr int cK = 0, cS = 2 * NG * 64, cO = cS + 2 * N;
    static_assert(cO + NG * N <= 512, "tensor memory");
    static_assert(kSmem <= 232448, "shared memory");
};

// One expander thread's cache row of the tiles ahead. The block number of the next tile is loaded a tile before it is used, in
// straight-line code (a load under a branch would be waited for where the branch ends).
struct Fetch {
    Cursor c;
    const uint8_t *codes;  // the cache, at the unit's first group
    const __half *norms;
    uint32_t g0, ng;
    int blk, off;
    bool ok, more;
};

template <bool KEYS>
__device__ __forceinline__ void fetch_unit(const TreeParams &p, Fetch &f) {
    const TreeUnit &u = p.unit[f.c.u];
    const int w = KEYS ? p.wk : p.wv, groups = KEYS ? p.kgroups : p.vgroups;
    const uint8_t *cache = KEYS ? p.t.k_cache : p.t.v_cache;
    f.g0 = KEYS ? u.gk : u.gv;
    f.ng = KEYS ? u.ngk : u.ngv;
    f.codes = cache + f.g0 * 16 * w;
    f.norms = reinterpret_cast<const __half *>(cache + (size_t)p.t.cap * ((size_t)groups * 16 * w));
}

__device__ __forceinline__ void fetch_block(const TreeParams &p, Fetch &f, int row) {
    const int t = f.c.tile * kTile + row, tc = max(0, min(t, f.c.len - 1));
    const int b = (int)((uint64_t)(uint32_t)tc * p.div_mul >> p.div_shift);  // tc / block_size
    f.off = tc - b * p.t.block_size;
    f.ok = t < f.c.len;
    f.blk = p.t.block_table[f.c.s * p.t.table_stride + b];  // b < max_blocks: len is cut to the table
}

// Starts the copies of the row's codes and norms; the norm's half of its word in `odd`.
template <int NG, bool KEYS, int W>
__device__ __forceinline__ bool fetch_codes(const TreeParams &p, const Fetch &f, uint32_t ring, uint32_t norm, int row, uint32_t &odd) {
    const int groups = KEYS ? p.kgroups : p.vgroups;
    const long long r = (long long)f.blk * p.t.block_size + f.off;
    bool ok = f.ok;
    if (ok && (f.blk < 0 || r >= p.t.cap)) {
        ok = false;
        atomicOr(p.status, kStatusIndex);
    }
    const size_t at0 = (size_t)r * groups + f.g0;
    odd = (uint32_t)at0 & 1;
    if (!ok) return false;
    const uint8_t *src = f.codes + (size_t)r * (groups * 16 * W);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        if (g == 1 && f.ng == 1) break;
        const uint32_t nd = norm + (g * kTile + row) * 4;
        const uint32_t dst = ring + (g * 4 * kTile + row) * 16;
#pragma unroll
        for (int i = 0; i < W; ++i) cp_async16(dst + i * kTile * 16, src + g * 16 * W + 16 * i);
        // the norm as the 4-byte word that holds it, unless that word would end past the cache
        const size_t at = at0 + g;
        if ((at | 1) < (size_t)p.t.cap * groups) cp_async4(nd, f.norms + (at & ~(size_t)1));
        else sts32(nd, (uint32_t)__half_as_ushort(f.norms[at]));
    }
    return true;
}
__device__ __forceinline__ float norm_value(uint32_t word, uint32_t odd) {
    return __half2float(__ushort_as_half((unsigned short)(odd ? word >> 16 : word)));
}

// The two products of tile i, issued by one warp. `first`: the tile starts its item's part.
template <int N, int NG>
__device__ __forceinline__ void issue_scores(const TreeParams &p, Shared &sh, uint8_t *smem, long long i, bool two) {
    using L = Plan<N, NG>;
    const int b = (int)(i & 1);
    const uint32_t par = (uint32_t)(i >> 1) & 1, tmem = sh.tmem;
    const uint64_t dz = desc_sw128(smem_u32(smem + L::oZ), 16);
    __syncwarp();
    wait(sh, &sh.k_full[b], par, p.status, 0x47490004u);
    wait(sh, &sh.s_empty[b], par ^ 1, p.status, 0x47490005u);
    fence_after();
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        if (g == 1 && !two) break;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            mma_ts(tmem + L::cS + b * N, tmem + L::cK + (b * NG + g) * 64 + 8 * k,
                   dz + (uint64_t)((g * L::kZBytes + (k >> 2) * (N * 128) + (k & 3) * 32) >> 4), idesc_f16(128, N, 0, 0), (g | k) != 0);
    }
    mma_commit(&sh.k_empty[b]);
    mma_commit(&sh.s_full[b]);
}
template <int N, int NG>
__device__ __forceinline__ void issue_sums(const TreeParams &p, Shared &sh, uint8_t *smem, long long i, bool first, bool two) {
    using L = Plan<N, NG>;
    const int b = (int)(i & 1), vb = L::kVBuf == 2 ? b : 0;
    const uint32_t par = (uint32_t)(i >> 1) & 1, tmem = sh.tmem;
    wait(sh, &sh.v_full[vb], L::kVBuf == 2 ? par : (uint32_t)(i & 1), p.status, 0x47490007u);
    wait(sh, &sh.p_full[b], par, p.status, 0x47490008u);
    fence_after();
    const uint64_t dp = desc_sw128(smem_u32(smem + L::oP) + b * L::kPBytes, kTile * 128);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        if (g == 1 && !two) break;
        const uint64_t dv = desc_sw128(smem_u32(smem + L::oV) + (vb * NG + g) * L::kVBytes, kTile * 128);
#pragma unroll
        for (int k = 0; k < 8; ++k)  // 16 cache rows: two atoms
            mma_ss(tmem + L::cO + g * N, dv + (uint64_t)(k * 2048 >> 4), dp + (uint64_t)(k * 2048 >> 4), idesc_f16(128, N, 1, 1),
                   !first || k);
    }
    mma_commit(&sh.v_empty[vb]);
    mma_commit(&sh.p_empty[b]);
}

// One side's expander warps: keys into tensor memory, values into shared memory.
template <int N, int NG, bool KEYS, int W>
__device__ void expand_role(const TreeParams &p, Shared &sh, uint8_t *smem, int row, int q, int lane) {
    using L = Plan<N, NG>;
    const uint32_t ring0 = smem_u32(smem + L::oRing) + (KEYS ? 0 : L::kDepth * L::kRing);
    const uint32_t norm0 = smem_u32(smem + L::oNorm) + (KEYS ? 0 : L::kDepth * L::kNorm);
    uint32_t tab[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) tab[i] = KEYS ? p.tk[i] : p.tv[i];
    Fetch f;
    f.c = sh.start;
    f.more = true;
    const long long tiles = f.c.left;
    fetch_unit<KEYS>(p, f);
    fetch_block(p, f, row);
    // per ring stage: the cache row exists; half of the first norm's word; the tile starts or ends its item's part; second group
    uint32_t valid = 0, odd = 0, starts = 0, ends = 0, has2 = 0;
    bool item_starts = true;
    int fs = 0;
    uint32_t zpar = 0;                    // warp 8: parity of the next item's queries
    bool owed = false, first_b = false, two_b = false;  // warp 12: the tile before waits for its sums
    auto fetch = [&]() {
        if (f.more) {
            uint32_t o;
            const bool ok = fetch_codes<NG, KEYS, W>(p, f, ring0 + fs * L::kRing, norm0 + fs * L::kNorm, row, o);
            const uint32_t bit = 1u << fs;
            const int u = f.c.u;
            f.more = f.c.advance(p, N);
            const bool next_starts = f.c.tile == 0;
            valid = ok ? valid | bit : valid & ~bit;
            odd = o ? odd | bit : odd & ~bit;
            starts = item_starts ? starts | bit : starts & ~bit;
            ends = next_starts || !f.more ? ends | bit : ends & ~bit;
            if (NG == 2) has2 = f.ng == 2 ? has2 | bit : has2 & ~bit;
            item_starts = next_starts;
            if (f.c.u != u) fetch_unit<KEYS>(p, f);
        }
        if (f.more) fetch_block(p, f, row);
        cp_commit();
        fs = fs + 1 == L::kDepth ? 0 : fs + 1;
    };
#pragma unroll 1
    for (int i = 0; i < L::kDepth; ++i) fetch();
    int rs = 0;
#pragma unroll 1
    for (long long i = 0; i < tiles; ++i) {
        const int b = (int)(i & 1);
        const uint32_t par = (uint32_t)(i >> 1) & 1;
        cp_wait<L::kDepth - 1>();
        const uint32_t ring = ring0 + rs * L::kRing, norm = norm0 + rs * L::kNorm;
        const uint32_t o0 = odd >> rs & 1;
        const uint32_t w0 = lds32(norm + row * 4);
        float n0 = norm_value(w0, o0), n1 = 0.0f;
        const bool none = !(valid >> rs & 1);
        const bool two = NG == 2 && (has2 >> rs & 1);
        if (NG == 2 && two) n1 = norm_value(lds32(norm + (kTile + row) * 4), o0 ^ 1);
        // Two groups with norms n0, n1: the product takes the larger one, the other group's levels are scaled by their ratio.
        float nn = n0, ratio[2] = {1.0f, 1.0f};
        uint32_t flip[2] = {0, 0};
        if (KEYS) {
            if (NG == 2 && two) {
                nn = fmaxf(fabsf(n0), fabsf(n1));
                ratio[0] = n0 / nn, ratio[1] = n1 / nn;
            }
        } else {
            nn = fabsf(n0);
            if (n0 < 0.0f) flip[0] = 0x80808080u;  // a negative norm turns its levels round
            if (NG == 2 && two) {
                if (n1 < 0.0f) flip[1] = 0x80808080u;
                nn = fmaxf(nn, fabsf(n1));
                ratio[0] = fabsf(n0) / nn, ratio[1] = fabsf(n1) / nn;
            }
        }
        if (NG == 2 && two) {
            const bool odd_norm = !(fabsf(n0) <= 65504.0f && fabsf(n1) <= 65504.0f);
            if (odd_norm) nn = __int_as_float(0x7FC00000);  // the row is lost for who attends it, and only for them
#pragma unroll
            for (int g = 0; g < 2; ++g)
                if (!(fabsf(ratio[g]) <= 1.0f)) ratio[g] = odd_norm ? 1.0f : 0.0f;  // 0/0: both norms are zero
        }
        wait(sh, &sh.s_empty[b], par ^ 1, p.status, 0x47490001u);
        if (KEYS) {
            sh.scal[b][0][row] = none ? 0.0f : nn;
        } else {
            // a norm of zero counts in the denominator: 2^-40 stands for it, far below the smallest fp16 norm
            const float safe = nn == 0.0f ? 0x1p-40f : nn;
            sh.scal[b][1][row] = none ? -INFINITY : nn <= 65504.0f ? log2f(safe) : __int_as_float(0x7FC00000);
            sh.scal[b][2][row] = !none && nn <= 65504.0f ? 1.0f / safe : 0.0f;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.sc_full[b]);
        const int vb = KEYS || L::kVBuf == 2 ? b : 0;
        const uint32_t vpar = KEYS || L::kVBuf == 2 ? par : (uint32_t)(i & 1);
        if (KEYS) {
            wait(sh, &sh.k_empty[b], par ^ 1, p.status, 0x47490002u);
            fence_after();
        } else {
            wait(sh, &sh.v_empty[vb], vpar ^ 1, p.status, 0x47490003u);
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            if (g == 1 && !two) break;
            uint32_t t[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) t[j] = KEYS || j < 4 ? tab[j] : tab[j] ^ flip[g];
            uint32_t c[4 * W];
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const uint4 v = lds128(ring + ((g * 4 + j) * kTile + row) * 16);
                c[4 * j] = v.x, c[4 * j + 1] = v.y, c[4 * j + 2] = v.z, c[4 * j + 3] = v.w;
            }
            const __half2 r2 = __float2half2_rn(ratio[g]);
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                uint32_t r[16];
                expand_quarter<W>(c + h * W, t, r);
                if (NG == 2) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        __half2 x = __hmul2(*reinterpret_cast<__half2 *>(&r[j]), r2);
                        r[j] = *reinterpret_cast<uint32_t *>(&x);
                    }
                }
                if (KEYS) {
                    tmem_st16(sh.tmem + ((uint32_t)(32 * q) << 16) + L::cK + (b * NG + g) * 64 + h * 16, r);
                } else {
                    // row `row` of the tile: two 64-wide segments of swizzled 16-byte chunks
                    const uint32_t base = smem_u32(smem + L::oV) + (vb * NG + g) * L::kVBytes + (h >> 1) * (kTile * 128) +
                                          (row >> 3) * 1024 + (row & 7) * 128;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        sts128(base + ((((h & 1) * 4 + j) ^ (row & 7)) << 4), r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
                }
            }
        }
        if (KEYS) {
            wait_st();
            fence_before();
        } else {
            fence_async();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(KEYS ? &sh.k_full[b] : &sh.v_full[vb]);
        // The products. The second one of a tile is issued an expansion later, when its weights are there, but at
        // once where the item's part ends, for its partials wait for it.
        if (q == 0) {
            const bool first = starts >> rs & 1;
            if (KEYS) {
                if (first) {
                    wait(sh, &sh.z_full, zpar, p.status, 0x47490006u);
                    zpar ^= 1;
                }
                issue_scores<N, NG>(p, sh, smem, i, two);
            } else {
                if (owed) issue_sums<N, NG>(p, sh, smem, i - 1, first_b, two_b);
                owed = !(ends >> rs & 1);
                if (!owed) issue_sums<N, NG>(p, sh, smem, i, first, two);
                first_b = first, two_b = two;
            }
            __syncwarp();
        }
        rs = rs + 1 == L::kDepth ? 0 : rs + 1;
        fetch();
    }
    if (q == 0) {  // MMAs in flight finish before tensor memory is freed
        mma_commit(&sh.drain[KEYS]);
        for (unsigned k = 0; k < kSpin; ++k)
            if (mbar_try(&sh.drain[KEYS], 0)) break;
        __syncwarp();
    }
    cp_wait<0>();
}

template <int N, int NG, bool KEYS>
__device__ void expand_any(const TreeParams &p, Shared &sh, uint8_t *smem, int row, int q, int lane) {
    switch (KEYS ? p.wk : p.wv) {
    case 2: expand_role<N, NG, KEYS, 2>(p, sh, smem, row, q, lane); break;
    case 3: expand_role<N, NG, KEYS, 3>(p, sh, smem, row, q, lane); break;
    default: expand_role<N, NG, KEYS, 4>(p, sh, smem, row, q, lane); break;
    }
}

// 128-point Sylvester transform over a warp, coordinates 4 * lane + j, unscaled.
__device__ __forceinline__ void fwht(float (&x)[4], int lane) {
    const float a = x[0] + x[1], b = x[0] - x[1], c = x[2] + x[3], d = x[2] - x[3];
    x[0] = a + c, x[1] = b + d, x[2] = a - c, x[3] = b - d;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float y = __shfl_xor_sync(0xFFFFFFFFu, x[j], o);
            x[j] = (lane & o) ? y - x[j] : x[j] + y;
        }
    }
}

__device__ __forceinline__ float load_q(const TreeParams &p, int64_t at) {
    return p.t.dtype == CQ_T_F16 ? __half2float(static_cast<const __half *>(p.t.q)[at])
                                 : __bfloat162float(static_cast<const __nv_bfloat16 *>(p.t.q)[at]);
}

// Rotated queries of an item's columns into shared memory (the K-major B operand), scaled by one power of two so that
// fp16 holds them whatever their size; returns what takes the scale back out of the logits.
template <int N, int NG>
__device__ float rotate_queries(const TreeParams &p, Shared &sh, uint8_t *smem, const Cursor &c, int warp, int lane) {
    using L = Plan<N, NG>;
    const TreeUnit &u = p.unit[c.u];
    const int rows = u.nh * p.per, cols = min(N, c.n * rows - c.c * N);
    float z[N / 8][NG][4], top = 0.0f;
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
        const int col = warp + 8 * i;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
#pragma unroll
            for (int j = 0; j < 4; ++j) z[i][g][j] = 0.0f;
            if (col < cols && g < u.ngk) {
                const int at = c.c * N + col, node = at / rows, r = at - node * rows, h = u.h0 + r / p.per;
                const int64_t src = (int64_t)(c.first + node) * p.t.q_stride_t + (int64_t)(u.h0 * p.per + r) * p.t.q_stride_h;
                const int d0 = (u.gk + g) * kGroup + 4 * lane - h * p.dk;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (d0 + j >= 0 && d0 + j < p.dk) z[i][g][j] = load_q(p, src + d0 + j);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < N / 8; ++i)
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            fwht(z[i][g], lane);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float a = fabsf(z[i][g][j]);
                if (a <= 3e38f) top = fmaxf(top, a);  // a lost column does not scale the others
            }
        }
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    if (lane == 0) atomicMax(&sh.zmax, __float_as_int(top));
    bar_sync(1, kSoftThreads);
    // largest coordinate between 2^13 and 2^14; the exponent is held where both powers of two are normal
    const int ex = max(-110, min(110, ((sh.zmax >> 23) & 255) - 127 - 13));
    const float down = __int_as_float((127 - ex) << 23);
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
        const int col = warp + 8 * i;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const uint32_t base = smem_u32(smem + L::oZ) + g * L::kZBytes + (col >> 3) * 1024 + (col & 7) * 128;
            auto put = [&](int pos, float x, float y) {
                const __half2 v = __floats2half2_rn(x * down, y * down);
                sts32(base + (pos >> 6) * (N * 128) + ((((pos & 63) >> 3) ^ (col & 7)) << 4) + (pos & 7) * 2,
                      *reinterpret_cast<const uint32_t *>(&v));
            };
            if (p.wk == 2) {
                put(position_of(4 * lane, 2), z[i][g][0], z[i][g][2]);
                put(position_of(4 * lane + 1, 2), z[i][g][1], z[i][g][3]);
            } else {
                put(4 * lane, z[i][g][0], z[i][g][1]);
                put(4 * lane + 2, z[i][g][2], z[i][g][3]);
            }
        }
    }
    return p.k_mult * __int_as_float((127 + ex) << 23);
}

// Who attends drafted token j, as bits over the item's columns.
template <int N>
__device__ void gather_mask(const TreeParams &p, Shared &sh, const Cursor &c, int warp, int lane) {
    const int rows = p.unit[c.u].nh * p.per, jw = (c.n + 31) / 32;
    for (int k = warp; k < jw * ((N + 31) / 32); k += 8) {
        const int cw = k / jw, j0 = (k - cw * jw) * 32, node = (c.c * N + cw * 32 + lane) / rows;
        uint32_t w = 0;
        if (node < c.n) {
            if (p.t.mask) w = p.t.mask[(int64_t)(c.first + node) * p.t.mask_words + (j0 >> 5)];
            else w = node >= j0 + 31 ? 0xFFFFFFFFu : node < j0 ? 0u : (2u << (node - j0)) - 1u;
        }
        uint32_t mine = 0;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const uint32_t v = __ballot_sync(0xFFFFFFFFu, w >> j & 1);
            if (lane == j) mine = v;
        }
        sh.mask[j0 + lane][cw] = mine;
    }
}

__device__ __forceinline__ int ordered(float x) {  // integers in the order of the floats
    const int i = __float_as_int(x);
    return i ^ ((i >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float unordered(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7FFFFFFF)); }

template <int N, int NG>
__device__ void softmax_role(const TreeParams &p, Shared &sh, uint8_t *smem, int warp, int lane) {
    using L = Plan<N, NG>;
    constexpr int NC = N / 2;                  // columns of this warpgroup
    constexpr int X = NC < 32 ? NC : 32;       // columns per tensor memory load
    const int wg = warp >> 2, q = warp & 3, row = 32 * q + lane, c0 = wg * NC;
    const uint32_t tm = sh.tmem + ((uint32_t)(32 * q) << 16);
    Cursor c = sh.start;
    long long i = 0, done = sh.w0;  // tiles done by this block; of all blocks
    bool more = true;
    while (more) {
        // ------------------------------------------------ one item's part --
        bar_sync(1, kSoftThreads);  // the item before is finished: zmax, m, mask may be written
        if (warp == 0 && lane == 0) sh.zmax = 0;
        if (lane + 32 * q < NC) sh.m[c0 + lane + 32 * q] = kNoMax;
        gather_mask<N>(p, sh, c, warp, lane);
        bar_sync(1, kSoftThreads);
        const float mult = rotate_queries<N, NG>(p, sh, smem, c, warp, lane);
        fence_async();
        fence_before();  // tensor memory reads of the item before
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.z_full);
        const TreeUnit u = p.unit[c.u];
        const int cols = min(N, c.n * u.nh * p.per - c.c * N), slot = blockIdx.x + c.item;
        const int i0 = (c.s * p.n_units + c.u) * p.ncol_max + c.c;
        if (c.tile == 0 && warp == 0 && lane == 0)
            p.rec[i0] = make_int2(slot, run_of(sh.total, p.grid, done + c.ntiles - 1) - (int)blockIdx.x + 1);
        const int count = (int)min((long long)(c.ntiles - c.tile), c.left);
        float l[NC];
#pragma unroll
        for (int k = 0; k < NC; ++k) l[k] = 0.0f;
#pragma unroll 1
        for (int it = 0; it < count; ++it, ++i) {
            const int b = (int)(i & 1);
            const uint32_t par = (uint32_t)(i >> 1) & 1;
            const int tok = (c.tile + it) * kTile;
            const bool masked = tok + kTile > c.ctx;  // the tile holds drafted tokens
            uint32_t see[(NC + 31) / 32];
#pragma unroll
            for (int k = 0; k < (NC + 31) / 32; ++k) {
                const int j = tok + row - c.ctx;
                see[k] = j >= 0 && j < c.n ? sh.mask[j][(c0 + 32 * k) >> 5] >> (c0 & 31) : 0xFFFFFFFFu;
            }
            wait(sh, &sh.sc_full[b], par, p.status, 0x47490009u);
            const float nk = sh.scal[b][0][row] * mult, ln = sh.scal[b][1][row], inv = sh.scal[b][2][row];
            wait(sh, &sh.s_full[b], par, p.status, 0x4749000Au);
            fence_after();
            // Column by column in halves of X: the denominators of all columns and the logits of one half fit the registers.
#pragma unroll
            for (int hf = 0; hf < NC; hf += X) {
                float d[X];
                const int cx = c0 + hf;
                const uint32_t ts = tm + L::cS + b * N + cx;
                auto logits = [&]() {  // d = log2 of the weights, before the reference
                    tmem_ld<X>(ts, d);
                    wait_ld<X>(d);
                    if (masked) {
#pragma unroll
                        for (int k = 0; k < X; ++k) {
                            const float x = fmaf(d[k], nk, ln);
                            d[k] = see[hf / 32] >> k & 1 ? x : -INFINITY;
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < X; ++k) d[k] = fmaf(d[k], nk, ln);
                    }
                };
                auto minus_reference = [&]() {
#pragma unroll
                    for (int k = 0; k < X; k += 4) {
                        const float4 m = *reinterpret_cast<const float4 *>(&sh.m[cx + k]);
                        d[k] -= m.x, d[k + 1] -= m.y, d[k + 2] -= m.z, d[k + 3] -= m.w;
                    }
                };
                logits();
                minus_reference();
                float top = d[0];
#pragma unroll
                for (int k = 1; k < X; ++k) top = fmaxf(top, d[k]);
                if (bar_or(2 + wg, 128, top > kRaise)) {
                    // ---------------------------------- raise references --
                    logits();
                    float mine = 0.0f;
#pragma unroll
                    for (int k = 0; k < X; ++k) {
                        const float x = unordered(__reduce_max_sync(0xFFFFFFFFu, ordered(fmaxf(d[k], -INFINITY))));
                        if (lane == k) mine = x;
                    }
                    if (lane < X) sh.wmax[warp][lane] = mine;
                    bar_sync(2 + wg, 128);
                    bool raised = false;
                    if (row < X) {
                        const float old = sh.m[cx + row];
                        float x = sh.wmax[4 * wg][row];
#pragma unroll
                        for (int k = 1; k < 4; ++k) x = fmaxf(x, sh.wmax[4 * wg + k][row]);
                        raised = x > old + kRaise;
                        sh.f[cx + row] = raised ? ex2(old - x) : 1.0f;
                        if (raised) sh.m[cx + row] = x;
                    }
                    raised = bar_or(2 + wg, 128, raised);
                    minus_reference();
                    if (raised) {
#pragma unroll
                        for (int k = 0; k < X; ++k) l[hf + k] *= sh.f[cx + k];
                        if (it) {  // the first tile's product does not accumulate
                            wait(sh, &sh.p_empty[b ^ 1], (uint32_t)((i - 1) >> 1) & 1, p.status, 0x4749000Bu);
                            fence_after();
                            for (int g = 0; g < u.ngv; ++g) {
#pragma unroll 1
                                for (int k = 0; k < X; k += 8) {
                                    float o[8];
                                    const uint32_t to = tm + L::cO + g * N + cx + k;
                                    tmem_ld<8>(to, o);
                                    wait_ld<8>(o);
#pragma unroll
                                    for (int j = 0; j < 8; ++j) o[j] *= sh.f[cx + k + j];
                                    tmem_st8(to, o);
                                }
                            }
                            wait_st();
                        }
                    }
                }
                if (hf + X == NC) {
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.s_empty[b]);
                }
                if (hf == 0) wait(sh, &sh.p_empty[b], par ^ 1, p.status, 0x4749000Cu);
                // weights in fp16: cache row `row`, columns cx .. cx + X - 1 (the MN-major B operand)
                const uint32_t pb = smem_u32(smem + L::oP) + b * L::kPBytes + (cx >> 6) * (kTile * 128) + (row >> 3) * 1024 + (row & 7) * 128;
#pragma unroll
                for (int k = 0; k < X; k += 8) {
                    uint32_t h[4];
#pragma unroll
                    for (int j = 0; j < 8; j += 2) {
                        const float x = ex2(d[k + j]), y = ex2(d[k + j + 1]);
                        l[hf + k + j] = fmaf(x, inv, l[hf + k + j]);
                        l[hf + k + j + 1] = fmaf(y, inv, l[hf + k + j + 1]);
                        const __half2 v = __floats2half2_rn(x, y);
                        h[j >> 1] = *reinterpret_cast<const uint32_t *>(&v);
                    }
                    sts128(pb + (((((cx + k) & 63) >> 3) ^ (row & 7)) << 4), h[0], h[1], h[2], h[3]);
                }
            }
            fence_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.p_full[b]);
        }
        // ------------------------------------------------- the item's partials --
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            float x = l[k];
#pragma unroll
            for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
            if (lane == 0) sh.lsum[warp][k] = x;
        }
        bar_sync(2 + wg, 128);
        if (row < NC && c0 + row < cols) {
            const float x = sh.lsum[4 * wg][row] + sh.lsum[4 * wg + 1][row] + (sh.lsum[4 * wg + 2][row] + sh.lsum[4 * wg + 3][row]);
            p.ml[(size_t)slot * N + c0 + row] = make_float2(sh.m[c0 + row], x);
        }
        wait(sh, &sh.p_empty[(i - 1) & 1], (uint32_t)((i - 1) >> 1) & 1, p.status, 0x4749000Du);
        fence_after();
        const int nat = natural_of(row, p.wv);
        for (int g = 0; g < u.ngv; ++g) {
            float *out = p.part + ((size_t)slot * NG + g) * N * kGroup + nat;
#pragma unroll
            for (int k = 0; k < NC; k += 8) {
                float o[8];
                tmem_ld<8>(tm + L::cO + g * N + c0 + k, o);
                wait_ld<8>(o);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c0 + k + j < cols) out[(size_t)(c0 + k + j) * kGroup] = o[j];
            }
        }
        done += count;
        c.left -= count;
        more = c.left > 0;
        if (more) c.next_item(p, N);
    }
}

template <int N, int NG>
__global__ void __launch_bounds__(kThreads, 1) tree_kernel(const __grid_constant__ TreeParams p) {
    using L = Plan<N, NG>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    Shared &sh = *reinterpret_cast<Shared *>(smem + L::oShared);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    if (tid == 0) {
        sh.abort = 0;
        sh.bad = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.k_full[i], 4);
            mbar_init(&sh.k_empty[i], 1);
            mbar_init(&sh.v_full[i], 4);
            mbar_init(&sh.v_empty[i], 1);
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.s_empty[i], 8);
            mbar_init(&sh.p_full[i], 8);
            mbar_init(&sh.p_empty[i], 1);
            mbar_init(&sh.sc_full[i], 8);
        }
        mbar_init(&sh.z_full, 8);
        mbar_init(&sh.drain[0], 1);
        mbar_init(&sh.drain[1], 1);
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    __syncthreads();
    const bool work = find_run<N>(p, sh);  // uniform
    if (blockIdx.x == 0 && tid == 0 && sh.bad) atomicOr(p.status, kStatusIndex);
    if (!work) return;
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(&sh.tmem)), "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::);
    }
    fence_before();
    __syncthreads();
    fence_after();
    // A softmax thread of many columns keeps logits and denominators in registers: the expanders give theirs up.
    // 256 (kSoft + kExp) = 512 x 128, what the block was launched with.
    if (warp < 8) {
        if (N >= 64) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(L::kSoft));
        softmax_role<N, NG>(p, sh, smem, warp, lane);
    } else if (warp < 12) {
        if (N >= 64) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(L::kExp));
        expand_any<N, NG, true>(p, sh, smem, tid - 256, warp & 3, lane);
    } else {
        if (N >= 64) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(L::kExp));
        expand_any<N, NG, false>(p, sh, smem, tid - 384, warp & 3, lane);
    }
    fence_before();
    __syncthreads();
    if (warp == 8) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(sh.tmem), "r"(512));
    }
}

// Joins the parts of an item, rotates and writes o. A block takes CG columns of an item: a warp per column
// where the parts are few, all warps on one column after the other where they are many.
constexpr int kJoinWarps = 8;
constexpr int kFewParts = 16;

template <int NG>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const __grid_constant__ TreeParams p, int N, int CG) {
    __shared__ float s_acc[kJoinWarps][NG][kGroup];
    __shared__ float2 s_ml[kJoinWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int item = blockIdx.x;
    const int s = item / (p.n_units * p.ncol_max), r0 = item - s * p.n_units * p.ncol_max, ui = r0 / p.ncol_max, ct = r0 - ui * p.ncol_max;
    const Seq q = seq_at(p, s);
    const TreeUnit &u = p.unit[ui];
    const int rows = u.nh * p.per, cols = min(N, q.n * rows - ct * N), first = blockIdx.y * CG;
    if (first >= cols) return;
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    const int2 rec = p.rec[item];
    const bool many = rec.y > kFewParts;
    for (int k = many ? 0 : warp; k < CG && first + k < cols; k += many ? 1 : kJoinWarps) {
        const int col = first + k;
        float M = kNoMax, sum = 0.0f, acc[NG][4];
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[g][j] = 0.0f;
        // the largest reference first (small loads), then the weighted sum in part order
        for (int a = lane; a < rec.y; a += 32) M = fmaxf(M, p.ml[(size_t)(rec.x + a) * N + col].x);
#pragma unroll
        for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
#pragma unroll 4
        for (int a = many ? warp : 0; a < rec.y; a += many ? kJoinWarps : 1) {
            const float2 ml = p.ml[(size_t)(rec.x + a) * N + col];
            const float w = ex2(ml.x - M);
            sum = fmaf(ml.y, w, sum);
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                if (g >= u.ngv) break;
                const float4 v = *reinterpret_cast<const float4 *>(p.part + (((size_t)(rec.x + a) * NG + g) * N + col) * kGroup + 4 * lane);
                acc[g][0] = fmaf(v.x, w, acc[g][0]), acc[g][1] = fmaf(v.y, w, acc[g][1]);
                acc[g][2] = fmaf(v.z, w, acc[g][2]), acc[g][3] = fmaf(v.w, w, acc[g][3]);
            }
        }
        if (many) {  // uniform in the block
            __syncthreads();
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int j = 0; j < 4; ++j) s_acc[warp][g][4 * lane + j] = acc[g][j];
            if (lane == 0) s_ml[warp] = make_float2(0.0f, sum);
            __syncthreads();
            if (warp) continue;
            sum = 0.0f;
            for (int w = 0; w < kJoinWarps; ++w) sum += s_ml[w].y;
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float x = 0.0f;
                    for (int w = 0; w < kJoinWarps; ++w) x += s_acc[w][g][4 * lane + j];
                    acc[g][j] = x;
                }
        }
        const int at = ct * N + col, node = at / rows, r = at - node * rows, h = u.h0 + r / p.per;
        const float f = sum == 0.0f ? 0.0f : p.v_mult / sum;  // zero: a token that attends nothing
        const int64_t dst = (int64_t)(q.first + node) * p.t.o_stride_t + (int64_t)(u.h0 * p.per + r) * p.t.o_stride_h;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            if (g >= u.ngv) break;
            fwht(acc[g], lane);
            const int d0 = (u.gv + g) * kGroup + 4 * lane - h * p.dv;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (d0 + j < 0 || d0 + j >= p.dv) continue;
                const float x = acc[g][j] * f;
                if (p.t.dtype == CQ_T_F16) static_cast<__half *>(p.t.o)[dst + d0 + j] = __float2half_rn(x);
                else static_cast<__nv_bfloat16 *>(p.t.o)[dst + d0 + j] = __float2bfloat16_rn(x);
            }
        }
    }
}

// ---------------------------------------------------------------------- host --
struct Shape {
    int n_units, ng, rows, N, ncol_max;
    size_t slots, items;
};

Shape shape_of(const cq_kv_geom &g, int n_seqs, int max_nodes, TreeUnit *u) {
    Shape s;
    s.n_units = tree_units(g, u);
    s.ng = 1;
    s.rows = 1;
    for (int i = 0; i < s.n_units; ++i) {
        s.ng = std::max<int>(s.ng, std::max(u[i].ngk, u[i].ngv));
        s.rows = std::max(s.rows, u[i].nh * (g.n_q_heads / g.n_kv_heads));
    }
    // The columns of a tile: what the largest tree needs, up to what tensor memory holds.
    const int most = s.rows * max_nodes, top = s.ng == 1 ? 128 : 64;
    s.N = 16;
    while (s.N < top && s.N < most) s.N *= 2;
    if (s.ng == 2 && s.N == 32) s.N = 64;
    s.ncol_max = std::max(1, (most + s.N - 1) / s.N);
    s.items = (size_t)n_seqs * s.n_units * s.ncol_max;
    s.slots = s.items + sm_count();
    return s;
}

size_t up16(size_t n) { return (n + 15) / 16 * 16; }

// Level tables as bytes, scaled by a power of two into [1, 2); returns that power.
float byte_table(const float *lv, uint32_t *t) {
    float top = 0.0f;
    for (int i = 0; i < 16; ++i) top = std::max(top, std::fabs(lv[i]));
    int e = 0;
    if (top > 0.0f) std::frexp(top, &e), --e;
    for (int i = 0; i < 8; ++i) t[i] = 0;
    for (int i = 0; i < 16; ++i) {
        const __half h = __float2half_rn(std::ldexp(lv[i], -e));
        const uint32_t b = __half_as_ushort(h);
        t[i / 4] |= (b & 255u) << (8 * (i & 3));
        t[4 + i / 4] |= (b >> 8) << (8 * (i & 3));
    }
    return std::ldexp(1.0f, e);
}

template <int N, int NG>
int launch_main(const TreeParams &p, cudaStream_t st) {
    const int rc = ensure_smem(reinterpret_cast<const void *>(tree_kernel<N, NG>), Plan<N, NG>::kSmem);
    if (rc) return rc;
    tree_kernel<N, NG><<<p.grid, kThreads, Plan<N, NG>::kSmem, st>>>(p);
    return CQ_OK;
}

}  // namespace

size_t tree_workspace(const cq_kv_geom &g, int n_seqs, int max_nodes) {
    if (!n_seqs || !max_nodes) return 0;
    TreeUnit u[kMaxUnits];
    const Shape s = shape_of(g, n_seqs, max_nodes, u);
    return up16(s.items * sizeof(int2)) + up16(s.slots * s.N * sizeof(float2)) + s.slots * s.ng * s.N * kGroup * sizeof(float);
}

int launch_kv_tree_attend(const cq_kv_geom &g, const cq_kv_tree &t, const float *lk, const float *lv, void *stream) {
    TreeParams p;
    const Shape s = shape_of(g, t.n_seqs, t.max_nodes, p.unit);
    if (s.slots > (size_t)INT_MAX / 2 || (s.N + 7) / 8 > 65535)
        return set_error(CQ_ERR_SHAPE, "%d requests of up to %d drafted tokens are too many for one call", t.n_seqs, t.max_nodes);
    p.t = t;
    p.n_units = s.n_units;
    p.hq = g.n_q_heads, p.per = g.n_q_heads / g.n_kv_heads, p.dk = g.head_dim_k, p.dv = g.head_dim_v;
    p.wk = width_of(g.k_bits), p.wv = width_of(g.v_bits);
    p.kgroups = in_padded(g.n_kv_heads * p.dk) / kGroup, p.vgroups = in_padded(g.n_kv_heads * p.dv) / kGroup;
    // t / block_size for t < 2^31: a product with 2^(31 + l) / block_size rounded up, 2^l >= block_size
    int l = 0;
    while (l < 31 && (1u << l) < (unsigned)t.block_size) ++l;
    p.div_shift = 31 + l;
    p.div_mul = (uint32_t)(((1ull << (31 + l)) + (unsigned)t.block_size - 1) / (unsigned)t.block_size);
    if (!t.max_blocks) p.t.block_table = t.cu_nodes, p.t.table_stride = 0;  // no token is read, but entry 0 is
    p.rows = s.rows, p.ncol_max = s.ncol_max, p.grid = sm_count();
    p.status = device_status_ptr();
    if (!p.status) return set_error(CQ_ERR_CUDA, "no device status word");
    uint8_t *ws = static_cast<uint8_t *>(t.workspace);
    p.rec = reinterpret_cast<int2 *>(ws);
    p.ml = reinterpret_cast<float2 *>(ws + up16(s.items * sizeof(int2)));
    p.part = reinterpret_cast<float *>(ws + up16(s.items * sizeof(int2)) + up16(s.slots * s.N * sizeof(float2)));
    p.k_mult = byte_table(lk, p.tk) * g.scale * 1.4426950408889634f * kInvSqrt128;
    p.v_mult = byte_table(lv, p.tv) * kInvSqrt128;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    int rc;
    if (s.ng == 1) {
        switch (s.N) {
        case 16: rc = launch_main<16, 1>(p, st); break;
        case 32: rc = launch_main<32, 1>(p, st); break;
        case 64: rc = launch_main<64, 1>(p, st); break;
        default: rc = launch_main<128, 1>(p, st); break;
        }
    } else {
        rc = s.N == 16 ? launch_main<16, 2>(p, st) : launch_main<64, 2>(p, st);
    }
    if (rc) return rc;
    // a block per column where there are few, eight columns otherwise
    const int cg = s.N == 16 ? 1 : 8;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)s.items, (unsigned)(s.N / cg));
    cfg.blockDim = dim3(32 * kJoinWarps);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess)
        e = s.ng == 1 ? cudaLaunchKernelEx(&cfg, join_kernel<1>, p, s.N, cg) : cudaLaunchKernelEx(&cfg, join_kernel<2>, p, s.N, cg);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return set_error(CQ_ERR_CUDA, "tree attention launch: %s", cudaGetErrorString(e));
    return CQ_OK;
}

}  // namespace cq
