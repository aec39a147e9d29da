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
// column's own logits it does not overflow whatever the size of the norms. m starts at the
// largest logit of 32 rows and rises when a column's w would pass 2^15 (the accumulators are then
// scaled, which is rare: at 2^8 it cost 5 to 9%); columns decide for themselves, so a column's bits do
// not depend on the others.
//
// Small weights. A w below 2^-14 loses bits in fp16 and one below 2^-25 is nothing, and the tensor core, too, drops what lies
// 2^-25 below its sum; the denominators keep them. One row far above all others would so cost a long context n 2^-25 of its
// result (0.38% of 131071 rows measured). Every kChunk tiles a part therefore starts over from references and sums of its own
// and is joined with what there was, in fp32: 16384 rows lose 2^-11 at most, one rounding of an fp16 result. It costs contexts
// of 65536 rows 1 to 4% (32 requests; 6% for single tokens of heads over two groups) and shorter parts nothing. (References
// below the largest logit keep such weights too, but rise often: 8 powers of two lower 314 -> 455 us for the server.)
//
// Queries in fp16. Each column is rounded at the power of two of its own largest element (rotate_queries), so that a query of any
// size leaves its tile mates' bits alone. The product then takes the columns at the tile's largest scale where that is exact for
// all of them, and else as they are, in which case softmax first multiplies their scores by their powers of two (scale_scores).
//
// Heads over two groups (a head of 96 or 256, say). Each group's levels are products of their own, and a row's two norms are
// n and r0 n, r1 n with the larger of them n: the scores stay apart in tensor memory until softmax adds them in fp32, while
// the values' levels are multiplied by their r in fp16, with one rounding.
//
// Split. The tiles of all (request, unit, column tile) items in one row are cut into equal runs, one per
// SM: lengths are read on the device, and the longest request cannot hold the launch up. Each run leaves
// unrotated partial sums; a second kernel joins them, rotates and writes o.
//
// Roles of the 16 or 20 warps. Softmax: one warpgroup, or two with half the columns each (N of 64 and
// more); they also rotate the queries and write the partials. Expansion: a warpgroup each for keys and
// values, in which a thread turns its cache row's codes into fp16 levels, keys into TMEM (the A operand)
// and values into shared memory. One warp issues the MMAs, two fetch codes, norms and block numbers into
// a ring some tiles ahead. Every wait is bounded: when one gives up, the flag `abort` makes all later
// waits return at once and every role runs through its remaining tiles without waiting, so that the
// block's barriers stay matched.
//
// What bounds it. Neither memory (18% of the copy rate for the decode batch below, which reads its caches once, 30% for the
// server, whose column tiles read them again: 602 MB for 198) nor the tensor pipe (22 to 36% of the dense
// rate at 128 columns): a tile of 16 columns takes about 2000 cycles and one of 128 about 3300, made of
// the latencies of five roles that hand each other buffers, with 46 to 51% of the issue slots used and
// shared memory busy for 45 to 66% of the time. An item (a request, unit and column tile) costs another
// 15000 to 20000 cycles to begin and end. Measured: 256 requests of 8000 tokens, 12 heads on 2 of 48/64, 2 bits,
// one token each, 117 us; 32 requests of 2000 to 8000 tokens with trees of 40 to 64, 32 heads on 8 of 128, 4 bits,
// 316 us; one of 131071 tokens with a tree of 64, the same heads, 2 bits, 205 us.
// Tried and slower: both sides or the keys alone looked up by byte permutes instead of tables (server 355 -> 495 us: the
// integer pipe runs at half rate), two expander warpgroups a side, two softmax streams or eight fetchers for 16
// columns (117 -> 120 to 145 us), leaving out the runs of 32 columns that a tree does not fill (203 -> 215 us and
// 313 -> 340 us: the branch keeps the two halves of a softmax thread's columns from overlapping).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstring>

#include "cq_paged.h"

namespace cq {
namespace {

constexpr int kTile = 128;        // cache rows per tile
constexpr int kMaxThreads = 640;
constexpr int kMaxDepth = 8;      // stages of the ring of codes
constexpr int kChunk = 128;       // tiles of an item that are summed from references of their own
constexpr unsigned kSpin = 1u << 20;   // polls of about 5 us each (measured)
constexpr float kNoMax = -1e30f;       // reference of a column that has attended nothing yet
constexpr float kRaise = 15.0f;         // log2 of the largest weight before a reference is raised (fp16 ends below 2^16)
constexpr float kInvSqrt128 = 0.08838834764831845f;
constexpr int kExLow = -110, kExHigh = 120;  // exponents of the queries' scales: both signs are normal powers of two
constexpr int kNoEx = -128;                 // of a column that is zero
constexpr int kGuard = 10;                   // a tile's columns share one scale where theirs are at most so many powers of two apart

struct TreeParams {
    cq_kv_tree t;
    TreeUnit unit[kMaxUnits];
    unsigned int *status;
    float *part;     // [slot][group][N][128] partial sums, unrotated
    float2 *ml;      // [slot][N] reference and denominator
    int2 *rec;       // [item] first slot and number of parts
    uint32_t tk[8], tv[8];  // level tables: low bytes of 16 fp16 levels, then high bytes
    float k_mult, v_mult;   // scale * log2(e) / sqrt(128) / (table scale); 1 / sqrt(128) / (table scale)
    int n_units, hq, per, dk, dv, wk, wv, kgroups, vgroups;
    int depth, stage;        // ring stages and their bytes
    uint32_t tab_k, tab_v;   // shared-memory addresses of the level tables
    uint32_t div_mul, div_shift;  // t / block_size = t * div_mul >> div_shift
    bool vec_q;      // a column's query is whole runs of 16 elements on 16-byte boundaries
    int rows;        // most query heads of a unit
    int slots;       // of part and ml
    unsigned spin;   // polls before a wait gives up
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
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity), "r"(1000u)
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
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// A value that every lane holds alike, in a form the compiler knows to be so.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xFFFFFFFFu, x, 0); }
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

// A tile in the row of all tiles.
struct Cursor {
    int s, u, c, tile, ntiles, ncol, first, n, ctx, len;
    int item;        // items before this one
    int left;        // tiles of this block's run from here on
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
    __device__ __forceinline__ bool advance(const TreeParams &p, int N) {  // to the next tile; false after the last
        if (--left <= 0) return false;
        if (++tile == ntiles) next_item(p, N);
        return true;
    }
};

// Beginning and ending an item takes a block as long as about this many tiles of N columns. They count as places in the row
// of tiles before the item's own, so that runs are equal in time (runs of equal tiles kept an SM busy 84% of the server's
// time and 94% of the decode batch's).
__host__ __device__ constexpr int item_cost(int N) { return N <= 32 ? 3 : 6; }

// Run b of `grid` blocks; with fewer places than blocks the first `total` blocks take one each, so that the parts of an
// item are consecutive blocks.
__device__ __forceinline__ long long run_start(long long total, int grid, int b) {
    const int n = (int)min(total, (long long)grid);
    if (b >= n) return total;
    return total < 1 << 21 ? (unsigned)total * (unsigned)b / (unsigned)n : total * b / n;  // grid < 2^11: a short division
}
__device__ __forceinline__ int run_of(long long total, int grid, long long tile) {
    return (int)(((tile + 1) * min(total, (long long)grid) - 1) / total);
}

struct Shared {
    uint64_t ring_full[kMaxDepth], ring_empty[kMaxDepth];
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], s_empty[2], sc_full[2], p_full, p_empty, z_full, drain;
    uint32_t tmem;
    volatile int abort;
    int ztop, zlow;               // largest and smallest exponent among the item's columns
    signed char zex[128];         // exponents of the columns' scales
    int bad;
    long long total, run[2];      // all places; this block's first one and the next block's
    long long first, edge[2];     // place of the first tile; tiles before this block's run and up to its end
    long long scan_t[kMaxThreads / 32];
    long long scan_i[kMaxThreads / 32];
    Cursor start;
    float scal[2][3][kTile];      // per tile buffer: n_k, log2 n_v, 1 / n_v
    alignas(16) float minus_m[128];  // column references, negated (read four at a time)
    alignas(16) float f[128];        // factors of the last raise
    float by_warp[8][64];         // column maxima of a softmax warp in a raise, denominators at an item's end
    uint32_t mask[CQ_TREE_MAX_NODES][4];  // columns (bits) that attend drafted token j
};

// The roles' loops run side by side on an SM and have to fit its instruction cache together (where they did not, each role
// waited for instructions most of the time): loops are kept rolled, and what runs once per item out of line.
__device__ __forceinline__ void wait(const TreeParams &p, Shared &sh, uint64_t *bar, uint32_t parity, unsigned code) {
    const uint32_t b = smem_u32(bar);
    for (unsigned i = 0; !mbar_try(b, parity) && !sh.abort; ++i)
        if (i >= p.spin) {
            atomicOr(p.status, code);
            sh.abort = 1;
        }
}

// Fills sh.start with this block's first tile and sh.total; false if it has no tile.
template <int N, int kThreads>
__device__ bool find_run(const TreeParams &p, Shared &sh) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kW = kThreads / 32;
    auto places_and_items = [&](int s, long long &t, long long &i) {
        t = i = 0;
        if (s >= p.t.n_seqs) return;
        const Seq q = seq_at(p, s);
        if (q.bad) sh.bad = 1;
        i = (long long)p.n_units * cols_of(p, q.n, N);
        t = q.n ? i * (tiles_of(q.len) + item_cost(N)) : 0;
    };
    // Inclusive sums of a and b up to this thread, and of all threads.
    auto scan = [&](long long a, long long b, long long &ia, long long &ib, long long &all_a, long long &all_b) {
        ia = a, ib = b;
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const long long ua = __shfl_up_sync(0xFFFFFFFFu, ia, o), ub = __shfl_up_sync(0xFFFFFFFFu, ib, o);
            if (lane >= o) ia += ua, ib += ub;
        }
        __syncthreads();
        if (lane == 31) sh.scan_t[warp] = ia, sh.scan_i[warp] = ib;
        __syncthreads();
        long long wa = lane < kW ? sh.scan_t[lane] : 0, wb = lane < kW ? sh.scan_i[lane] : 0;
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const long long ua = __shfl_up_sync(0xFFFFFFFFu, wa, o), ub = __shfl_up_sync(0xFFFFFFFFu, wb, o);
            if (lane >= o) wa += ua, wb += ub;
        }
        all_a = __shfl_sync(0xFFFFFFFFu, wa, 31), all_b = __shfl_sync(0xFFFFFFFFu, wb, 31);
        const long long pa = __shfl_sync(0xFFFFFFFFu, wa, max(warp - 1, 0)), pb = __shfl_sync(0xFFFFFFFFu, wb, max(warp - 1, 0));
        if (warp) ia += pa, ib += pb;
    };
    // The sum over all requests; those of the first chunk are kept.
    long long a, b, ia, ib, all_a, all_b, total = 0;
    places_and_items(tid, a, b);
    for (int s = tid + kThreads; s < p.t.n_seqs; s += kThreads) {
        long long x, y;
        places_and_items(s, x, y);
        total += x;
    }
    if (p.t.n_seqs > kThreads) {  // uniform
        scan(total, 0, ia, ib, all_a, all_b);
        total = all_a;
    }
    scan(a, b, ia, ib, all_a, all_b);
    total += all_a;
    if (tid < 2) sh.run[tid] = run_start(total, p.grid, blockIdx.x + tid);
    if (tid == 0) sh.total = total;
    __syncthreads();
    const long long w0 = sh.run[0], w1 = sh.run[1];
    if (w0 >= w1) return false;
    long long ct = 0, ci = 0;  // places and items before the chunk
    for (int base = 0;;) {
        const long long t0 = ct + ia - a;
#pragma unroll 1
        for (int e = 0; e < 2; ++e) {  // exactly one thread finds the run's first place, one its last
            const long long off = (e ? w1 - 1 : w0) - t0;
            if (off < 0 || off >= a) continue;
            Cursor c;
            c.s = base + tid;
            c.take(p, N);
            const int places = c.ntiles + item_cost(N);
            const int it = off < 1ll << 32 ? (int)((unsigned)off / (unsigned)places) : (int)(off / places);
            const int in = (int)(off - (long long)it * places) - item_cost(N);  // a tile, or below zero
            const long long item = ci + ib - b + it;
            sh.edge[e] = t0 + (long long)it * places - item * item_cost(N) + max(0, in + e);
            if (e) continue;
            c.tile = max(0, in);
            c.u = it / c.ncol;
            c.c = it - c.u * c.ncol;
            c.item = (int)item;
            sh.first = w0 + (c.tile - in);
            sh.start = c;
        }
        ct += all_a, ci += all_b;
        base += kThreads;
        if (ct >= w1 || base >= p.t.n_seqs) break;  // uniform
        places_and_items(base + tid, a, b);
        scan(a, b, ia, ib, all_a, all_b);
    }
    __syncthreads();
    if (tid == 0) sh.start.left = (int)(sh.edge[1] - sh.edge[0]);  // read after the next barrier
    return sh.edge[1] > sh.edge[0];
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
template <int N, int NG, int ZT>
struct Plan {
    static constexpr int kSoftWG = N >= 64 ? 2 : 1;              // warpgroups of softmax
    static constexpr int kSoft = 4 * kSoftWG, kExp = 8;         // warps; then the issuer, two fetchers, one idle
    static constexpr int kThreads = 32 * (kSoft + kExp + 4);
    static constexpr int kIssue = N <= 32 ? 4 : 1;               // MMAs in line: with few columns the issuer is the slowest role
    static constexpr int kVBuf = NG == 1 && !(N == 128 && ZT == 2) ? 2 : 1;
    static constexpr int kVBytes = 2 * kTile * 128;            // one group's values: 128 rows x 128 fp16
    static constexpr int kPBytes = kTile * (N <= 64 ? 128 : 256);
    static constexpr int kZBytes = N * 256;                    // one group
    // ZT: fp16 queries come rotated as a sum of two fp16 terms: one term would be the largest part of an fp16 result's error
    // (0.00048 against the 0.0002 of the result's own rounding). bf16 results do not show it. At 128 columns the second
    // term takes the place of the second buffer of values, in a kernel of its own.
    static constexpr int oV = 0, oP = oV + kVBuf * NG * kVBytes, oZ = oP + kPBytes, oShared = oZ + NG * ZT * kZBytes;
    static constexpr int oRatio = oShared + ((int)sizeof(Shared) + 127) / 128 * 128;  // per tile buffer and group: a row's key norms over the larger
    static constexpr int oRing = oRatio + (NG == 2 ? 2 * NG * kTile * 4 : 0);
    // registers of the roles where softmax takes two warpgroups: 256 (kSoftRegs + kExpRegs) + 128 kRestRegs <= 640 x 96
    static constexpr int kSoftRegs = N == 128 ? 144 : 128, kExpRegs = N == 128 ? 64 : 72, kRestRegs = N == 128 ? 64 : 80;
    // TMEM columns
    static constexpr int kKBuf = NG == 2 && N == 64 ? 1 : 2;     // 512 columns hold no second buffer of keys then
    static constexpr int cK = 0, cS = kKBuf * NG * 64, cO = cS + 2 * NG * N;
    static_assert(cO + NG * N <= 512, "tensor memory");
};

// A block's shared memory as addresses: the first kilobyte is the system's. The tables lie at the top, each aligned to its
// size, so that an entry's address is put together by one logical operation.
constexpr int kSmemFirst = 1024, kSmemLast = 232448 + 1024, kTabTop = kSmemLast / 32768 * 32768;

// Level tables in shared memory (one group per row): entry e at e * 128 bytes, repeated for every lane so that no two lanes of a
// warp meet in a bank. A code pair gives one fp16 pair (3 and 4 bits, and 2 bits where space is short), a byte of two-bit
// codes four levels. A pair costs two integer instructions and a load; byte permutes of register tables, on the half-rate
// integer pipe, bounded the kernel (407 -> 316 us and 903 -> 618 us for the long context and the server below, when this came).
__host__ __device__ constexpr bool wide_two(int N) { return N <= 32; }
__host__ __device__ constexpr int table_bytes(int w, int N) { return w == 4 || (w == 2 && wide_two(N)) ? 256 * 128 : w == 3 ? 64 * 128 : 16 * 128; }

// Two warps fetch: a lane has the cache rows `lane` and `lane + 64` of the tiles ahead. The block numbers of the next tile are loaded a
// tile before they are used, in straight-line code (a load under a branch would be waited for where the branch ends).
struct RowAt {
    int blk, off;
    bool ok;
};
__device__ __forceinline__ RowAt row_at(const TreeParams &p, const Cursor &c, int row) {
    RowAt r;
    const int t = c.tile * kTile + row, tc = max(0, min(t, c.len - 1));
    const int b = (int)((uint64_t)(uint32_t)tc * p.div_mul >> p.div_shift);  // tc / block_size
    r.off = tc - b * p.t.block_size;
    r.ok = t < c.len;
    r.blk = p.t.block_table[c.s * p.t.table_stride + b];  // b < max_blocks: len is cut to the table
    return r;
}

// A stage of the ring: codes of the keys as [group][16-byte chunk][row], then of the values; a word per row and side: bit 0 the
// row exists, bit 1 the half of the norm words that holds the first group's norm, bit 2 the norm itself is in the upper
// half (where the word would end past the cache); norm words as [side][group][row].
template <int NG>
struct Stage {
    static constexpr int kInfo = 2 * kTile * 4, kNorms = 2 * NG * kTile * 4;
    __host__ __device__ static constexpr int codes(int w) { return NG * w * kTile * 16; }
    __host__ __device__ static constexpr int bytes(int wk, int wv) { return codes(wk) + codes(wv) + kInfo + kNorms; }
};

// A side of the cache as the fetchers take it.
struct Side {
    const uint8_t *codes;  // at the unit's first group
    const __half *norms;   // likewise
    uint32_t stride, groups, g0, ng, w;
};
template <bool KEYS>
__device__ __forceinline__ Side side_of(const TreeParams &p, int unit) {
    Side s;
    const TreeUnit &u = p.unit[unit];
    s.g0 = KEYS ? u.gk : u.gv, s.ng = KEYS ? u.ngk : u.ngv;
    s.w = KEYS ? p.wk : p.wv, s.groups = KEYS ? p.kgroups : p.vgroups;
    s.stride = s.groups * 16 * s.w;
    const uint8_t *cache = KEYS ? p.t.k_cache : p.t.v_cache;
    s.codes = cache + s.g0 * 16 * s.w;
    s.norms = reinterpret_cast<const __half *>(cache + (size_t)p.t.cap * s.stride);
    return s;
}

template <int NG>
__device__ __forceinline__ void fetch_side(const Side &s, uint32_t r, size_t all, uint32_t codes, uint32_t info, uint32_t norms) {
    const uint8_t *src = s.codes + (size_t)r * s.stride;
    const size_t at = (size_t)r * s.groups + s.g0;
    uint32_t word = 1 | (uint32_t)(at & 1) << 1;
    const uint32_t chunks = NG == 2 ? s.ng * s.w : s.w;
#pragma unroll
    for (int i = 0; i < 4 * NG; ++i)
        if (i < chunks) cp_async16(codes + i * kTile * 16, src + i * 16);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        if (g >= s.ng) break;
        if (((at + g) | 1) < all) cp_async4(norms + g * kTile * 4, s.norms + ((at + g) & ~(size_t)1));
        else word |= 4 | (uint32_t)__half_as_ushort(s.norms[at + g]) << 16;  // the last norm of all: never the first of two
    }
    sts32(info, word);
}

template <int N, int NG, int ZT>
__device__ void fetch_role(const TreeParams &p, Shared &sh, uint8_t *smem, int lane) {
    using L = Plan<N, NG, ZT>;
    Cursor c = sh.start;
    const int tiles = uniform(c.left);
    const uint32_t ring = smem_u32(smem) + L::oRing;
    // block numbers of the next two halves; the cursor is a tile ahead of the copies
    RowAt next = row_at(p, c, lane), after = row_at(p, c, lane + 64);
    int st = 0, unit = c.u, unit_next = c.u;
    uint32_t par = 1;
    Side sk = side_of<true>(p, unit), sv = side_of<false>(p, unit);
    const size_t all_k = (size_t)p.t.cap * sk.groups, all_v = (size_t)p.t.cap * sv.groups;
#pragma unroll 1
    for (int i = 0; i < 2 * tiles; ++i) {  // half a tile at a time
        const int half = i & 1;
        if (!half) {
            if (unit_next != unit) {
                unit = unit_next;
                sk = side_of<true>(p, unit), sv = side_of<false>(p, unit);
            }
            c.advance(p, N);
            unit_next = c.u;
        }
        const RowAt now = next;
        next = after;
        after = row_at(p, c, lane + 64 * half);
        if (!half) wait(p, sh, &sh.ring_empty[st], par, 0x4749000Eu);
        const uint32_t kc = ring + st * p.stage + (lane + 64 * half) * 16, vc = kc + Stage<NG>::codes(p.wk);
        const uint32_t info = vc + Stage<NG>::codes(p.wv) - (lane + 64 * half) * 12, nrm = info + Stage<NG>::kInfo;
        const long long at = (long long)now.blk * p.t.block_size + now.off;
        const bool ok = now.ok && now.blk >= 0 && at < p.t.cap;
        if (ok) {
            fetch_side<NG>(sk, (uint32_t)at, all_k, kc, info, nrm);
            fetch_side<NG>(sv, (uint32_t)at, all_v, vc, info + kTile * 4, nrm + NG * kTile * 4);
        } else {
            sts32(info, 0);
            sts32(info + kTile * 4, 0);
            if (now.ok) atomicOr(p.status, kStatusIndex);
        }
        if (half) {
            // two arrivals a lane: one when its copies have landed, one for what it stored itself
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(smem_u32(&sh.ring_full[st])) : "memory");
            mbar_arrive(&sh.ring_full[st]);
            if (++st == p.depth) st = 0, par ^= 1;
        }
    }
    asm volatile("cp.async.wait_all;\n" ::: "memory");
}

// Norm of group g from a row's info and norm words (a norm given in the info word is that of the last group).
__device__ __forceinline__ float norm_value(uint32_t info, uint32_t word, int g, int last) {
    const uint32_t bits = info & 4 && g == last ? info >> 16 : ((info >> 1) + g) & 1 ? word >> 16 : word & 0xFFFFu;
    return __half2float(__ushort_as_half((unsigned short)bits));
}

// The two products of tile i, issued by one warp. `first`: the tile starts its item's part.
template <int N, int NG, int ZT>
__device__ __forceinline__ void issue_scores(const TreeParams &p, Shared &sh, uint8_t *smem, uint32_t tmem, int i, bool two) {
    using L = Plan<N, NG, ZT>;
    const int b = i & 1, kb = L::kKBuf == 2 ? b : 0;
    const uint32_t par = (uint32_t)(i >> 1) & 1;
    const uint64_t dz = desc_sw128(smem_u32(smem + L::oZ), 16);
    wait(p, sh, &sh.k_full[kb], L::kKBuf == 2 ? par : (uint32_t)(i & 1), 0x47490004u);
    wait(p, sh, &sh.s_empty[b], par ^ 1, 0x47490005u);
    __syncwarp();
    fence_after();
    // two groups keep their scores apart: their norms are ratios for softmax, which multiplies in fp32
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        if (g == 1 && !two) break;
#pragma unroll
        for (int t = 0; t < ZT; ++t) {
            if (t == 1 && N < 128 && p.t.dtype != CQ_T_F16) break;  // the second term of the queries
#pragma unroll L::kIssue
            for (int k = 0; k < 8; ++k)
                mma_ts(tmem + L::cS + (b * NG + g) * N, tmem + L::cK + (kb * NG + g) * 64 + 8 * k,
                       dz + (uint64_t)(((t * NG + g) * L::kZBytes + (k >> 2) * (N * 128) + (k & 3) * 32) >> 4), idesc_f16(128, N, 0, 0), (t | k) != 0);
        }
    }
    mma_commit(&sh.k_empty[kb]);
    mma_commit(&sh.s_full[b]);
}
template <int N, int NG, int ZT>
__device__ __forceinline__ void issue_sums(const TreeParams &p, Shared &sh, uint8_t *smem, uint32_t tmem, int i, bool first, bool two) {
    using L = Plan<N, NG, ZT>;
    const int vb = L::kVBuf == 2 ? i & 1 : 0;
    wait(p, sh, &sh.v_full[vb], L::kVBuf == 2 ? (uint32_t)(i >> 1) & 1 : (uint32_t)(i & 1), 0x47490007u);
    wait(p, sh, &sh.p_full, (uint32_t)(i & 1), 0x47490008u);
    __syncwarp();
    fence_after();
    const uint64_t dp = desc_sw128(smem_u32(smem + L::oP), kTile * 128);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        if (g == 1 && !two) break;
        const uint64_t dv = desc_sw128(smem_u32(smem + L::oV) + (vb * NG + g) * L::kVBytes, kTile * 128);
#pragma unroll L::kIssue
        for (int k = 0; k < 8; ++k)  // 16 cache rows: two atoms
            mma_ss(tmem + L::cO + g * N, dv + (uint64_t)(k * 2048 >> 4), dp + (uint64_t)(k * 2048 >> 4), idesc_f16(128, N, 1, 1),
                   !first || k);
    }
    mma_commit(&sh.v_empty[vb]);
    mma_commit(&sh.p_empty);
}

template <int N, int NG, int ZT>
__device__ void issue_role(const TreeParams &p, Shared &sh, uint8_t *smem) {
    Cursor c = sh.start;
    const uint32_t tmem = uniform(sh.tmem);
    const int tiles = uniform(c.left);
    uint32_t zpar = 0;
    bool next_first = true;  // tile i + 1 starts its item's part
    int since = 0;           // tiles of this part before tile i
#pragma unroll 1
    for (int i = 0; i < tiles; ++i) {
        const bool two_k = NG == 2 && uniform(p.unit[c.u].ngk == 2), two_v = NG == 2 && uniform(p.unit[c.u].ngv == 2);
        if (next_first) {
            wait(p, sh, &sh.z_full, zpar, 0x47490006u);
            zpar ^= 1;
            issue_scores<N, NG, ZT>(p, sh, smem, tmem, i, two_k);
            since = 0;
        }
        const bool first = since++ % kChunk == 0;  // of a chunk
        const bool more = c.advance(p, N);
        next_first = uniform(!more || c.tile == 0);
        if (!next_first) issue_scores<N, NG, ZT>(p, sh, smem, tmem, i + 1, two_k);  // while softmax works on tile i
        issue_sums<N, NG, ZT>(p, sh, smem, tmem, i, first, two_v);
    }
    mma_commit(&sh.drain);  // MMAs in flight finish before tensor memory is freed
    for (unsigned k = 0; k < kSpin; ++k)
        if (mbar_try(smem_u32(&sh.drain), 0)) break;
    __syncwarp();
}

// ------------------------------------------------------------- expansion --
// The W words of a row's quarter h (32 codes) from a ring stage.
template <int W>
__device__ __forceinline__ void load_quarter(uint32_t codes, int row, int h, uint32_t (&c)[W]) {
    if (W == 4) {
        const uint4 v = lds128(codes + (h * kTile + row) * 16);
        c[0] = v.x, c[1] = v.y, c[W - 2] = v.z, c[W - 1] = v.w;
    } else if (W == 2) {
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];\n" : "=r"(c[0]), "=r"(c[1]) : "r"(codes + ((h >> 1) * kTile + row) * 16 + (h & 1) * 8));
    } else {
#pragma unroll
        for (int k = 0; k < W; ++k) c[k] = lds32(codes + (((W * h + k) >> 2) * kTile + row) * 16 + ((W * h + k) & 3) * 4);
    }
}

// 32 codes in words c as 16 fp16 pairs in their order, from the table at `tab` (plus this lane's place in a row).
template <int N, int W>
__device__ __forceinline__ void lookup_quarter(const uint32_t (&c)[W], uint32_t tab, uint32_t (&r)[16]) {
    if (W == 2 && wide_two(N)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t x = c[j / 4];
            const int s = 8 * (j & 3) - 7;
            const uint32_t a = tab | ((s < 0 ? x << 7 : x >> (s < 0 ? 0 : s)) & 0x7F80u);
            asm("ld.shared.v2.u32 {%0, %1}, [%2];\n" : "=r"(r[2 * j]), "=r"(r[2 * j + 1]) : "r"(a));
        }
    } else {
        constexpr int kBits = 2 * W;
        constexpr uint32_t kMask = ((1u << kBits) - 1) << 7;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const int at = kBits * j, w = at / 32, s = at % 32;  // the pair's bits: from bit s of word w
            uint32_t x;
            if (s + kBits > 32) x = __funnelshift_r(c[w], c[w + 1 < W ? w + 1 : w], s) << 7;
            else x = s < 7 ? c[w] << (7 - s) : c[w] >> (s - 7);
            asm("ld.shared.u32 %0, [%1];\n" : "=r"(r[j]) : "r"(tab | (x & kMask)));  // the tables never change
        }
    }
}

// Fills a table (all threads); t: the levels' bytes as in TreeParams.
__device__ void fill_table(uint32_t dst, const uint32_t (&t)[8], int w, bool wide) {
    const int entries = w == 4 || wide ? 256 : w == 3 ? 64 : 16;
#pragma unroll 1
    for (int i = threadIdx.x; i < entries * 8; i += blockDim.x) {  // 16 bytes each
        const uint32_t e = i >> 3;
        uint32_t r[8], a, b;
        if (w == 2) {  // pairs of codes 0 and 2, .. of 1 and 3, ..
            expand_w2(e, t, r);
            a = prmt(r[0], r[4], 0x5410), b = wide ? prmt(r[0], r[4], 0x7632) : a;
        } else {
            if (w == 3) expand_w3(e, t, r);
            else expand_w4(e, t, r);
            a = b = r[0];
        }
        sts128(dst + i * 16, a, b, a, b);
    }
}

// Expander warps: keys into tensor memory, values into shared memory, and the rows' norms for softmax. One code for both sides.
template <int N, int NG, int ZT, int W>
__device__ __forceinline__ void expand_tile(const TreeParams &p, uint8_t *smem, uint32_t tmem, bool keys, uint32_t codes, uint32_t tab, int buf, int row,
                                            int q, const float (&ratio)[2], uint32_t flip, bool two) {
    using L = Plan<N, NG, ZT>;
#pragma unroll 1
    for (int g = 0; g < (two ? 2 : 1); ++g) {
        uint32_t t[8];
        if (NG == 2) {
#pragma unroll
            for (int j = 0; j < 8; ++j) t[j] = keys ? p.tk[j] : j < 4 ? p.tv[j] : p.tv[j] ^ (flip & 0x80808080u);
        }
        // the values' ratio as two fp16 terms: what is left is the product's one rounding
        const float ratio_g = NG == 2 && g ? ratio[1] : ratio[0];
        const __half2 r2 = __float2half2_rn(ratio_g), r2_low = __float2half2_rn(ratio_g - __low2float(r2));
        const bool turned = NG == 1 && __any_sync(0xFFFFFFFFu, flip != 0);
        const uint32_t from = codes + g * W * kTile * 16;
        const uint32_t to_k = tmem + ((uint32_t)(32 * q) << 16) + L::cK + (buf * NG + g) * 64;
        // row `row` of the tile: two 64-wide segments of swizzled 16-byte chunks
        const uint32_t to_v = smem_u32(smem + L::oV) + (buf * NG + g) * L::kVBytes + (row >> 3) * 1024 + (row & 7) * 128;
        uint32_t next[W];
        load_quarter<W>(from, row, 0, next);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            uint32_t r[16], c[W];
#pragma unroll
            for (int j = 0; j < W; ++j) c[j] = next[j];
            load_quarter<W>(from, row, min(h + 1, 3), next);
            if (NG == 1) {
                lookup_quarter<N, W>(c, tab, r);
            } else {
                expand_quarter<W>(c, t, r);
                // keys are not scaled; with few columns they go through the same code with a ratio of one (16 columns, four bits:
                // 210 us against 221 with a branch), with many the time counts (64 columns: 193 to 529 us against 207 to 542)
                if (N <= 32 || !keys) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const __half2 l = *reinterpret_cast<__half2 *>(&r[j]), x = __hfma2(l, r2, __hmul2(l, r2_low));
                        r[j] = *reinterpret_cast<const uint32_t *>(&x);
                    }
                }
            }
            if (keys) {
                tmem_st16(to_k + h * 16, r);
            } else {
                const uint32_t base = to_v + (h >> 1) * (kTile * 128);
                if (NG == 1 && __builtin_expect(turned, 0)) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) r[j] ^= flip;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    sts128(base + ((((h & 1) * 4 + j) ^ (row & 7)) << 4), r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
                }
            }
        }
    }
}

// The norm of a side's row, and for two groups of norms n0, n1 the larger one with each group's ratio to it, by which its levels
// are scaled. Ratios stay finite whatever the norms, so that a lost row reaches only who attends it.
template <int NG>
__device__ __forceinline__ float row_norm(uint32_t info, uint32_t norms, bool two, float (&ratio)[2]) {
    const float n0 = norm_value(info, lds32(norms), 0, NG == 2 && two ? 1 : 0);
    ratio[0] = ratio[1] = 1.0f;
    if (NG == 1 || !two) return n0;
    const float n1 = norm_value(info, lds32(norms + kTile * 4), 1, 1);
    float nn = fmaxf(fabsf(n0), fabsf(n1));
    const bool lost = !(fabsf(n0) <= 65504.0f && fabsf(n1) <= 65504.0f);
    ratio[0] = n0 / nn, ratio[1] = n1 / nn;
#pragma unroll
    for (int g = 0; g < 2; ++g)
        if (!(fabsf(ratio[g]) <= 1.0f)) ratio[g] = lost ? 1.0f : 0.0f;  // 0 / 0: both norms are zero
    return lost ? __int_as_float(0x7FC00000) : nn;
}

template <int N, int NG, int ZT>
__device__ void expand_role(const TreeParams &p, Shared &sh, uint8_t *smem, bool keys, int row, int q, int lane) {
    using L = Plan<N, NG, ZT>;
    Cursor c = sh.start;
    const int tiles = uniform(c.left), w = keys ? p.wk : p.wv;
    const uint32_t tmem = uniform(sh.tmem), ring = smem_u32(smem) + L::oRing;
    const uint32_t tab = (keys ? p.tab_k : p.tab_v) | (w == 2 && wide_two(N) ? (lane & 15) * 8 : lane * 4);
    int st = 0;
    uint32_t rpar = 0;
#pragma unroll 1
    for (int i = 0; i < tiles; ++i) {
        const bool twice = (keys ? L::kKBuf : L::kVBuf) == 2;
        const int b = i & 1, buf = twice ? b : 0;
        const uint32_t par = (uint32_t)(i >> 1) & 1;
        bool two = false;
        if (NG == 2) {
            two = (keys ? p.unit[c.u].ngk : p.unit[c.u].ngv) == 2;
            c.advance(p, N);
        }
        float ratio[2];
        uint32_t flip = 0;
        const uint32_t codes = ring + st * p.stage, info = codes + Stage<NG>::codes(p.wk) + Stage<NG>::codes(p.wv) + (keys ? 0 : kTile * 4);
        const uint32_t nrm = info + Stage<NG>::kInfo + (keys ? 0 : (NG - 1) * kTile * 4);
        wait(p, sh, &sh.ring_full[st], rpar, 0x4749000Fu);
        const uint32_t word = lds32(info + row * 4);
        float n = row_norm<NG>(word, nrm + row * 4, two, ratio);
        if (!keys) {
            if (!two) {
                if (n < 0.0f) flip = 0x80008000u;  // a negative norm turns its levels round
                if (NG == 2) flip |= flip >> 8;    // byte tables: the high bytes' signs
                n = fabsf(n);
            }
        }
        // a norm of zero counts in the denominator: 2^-40 stands for it, far below the smallest fp16 norm
        const float safe = n == 0.0f ? 0x1p-40f : n;
        const bool lost = !(n <= 65504.0f), real = word & 1;
        const float ln = lost ? __int_as_float(0x7FC00000) : __log2f(safe), inv = lost ? 0.0f : __fdividef(1.0f, safe);
        wait(p, sh, &sh.s_empty[b], par ^ 1, 0x47490001u);
        if (keys) {
            sh.scal[b][0][row] = real ? n : 0.0f;
            if (NG == 2) {  // softmax applies the ratios of the keys, in fp32
                const uint32_t to = smem_u32(smem + L::oRatio) + (b * 2 * kTile + row) * 4;
                sts32(to, __float_as_uint(ratio[0]));
                sts32(to + kTile * 4, __float_as_uint(ratio[1]));
                ratio[0] = ratio[1] = 1.0f;
            }
        } else {
            sh.scal[b][1][row] = real ? ln : -INFINITY;
            sh.scal[b][2][row] = real ? inv : 0.0f;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.sc_full[b]);
        wait(p, sh, keys ? &sh.k_empty[buf] : &sh.v_empty[buf], (twice ? par : (uint32_t)(i & 1)) ^ 1, 0x47490002u);
        fence_after();
        const uint32_t from = keys ? codes : codes + Stage<NG>::codes(p.wk);
        if (w == 2) expand_tile<N, NG, ZT, 2>(p, smem, tmem, keys, from, tab, buf, row, q, ratio, flip, two);
        else if (w == 3) expand_tile<N, NG, ZT, 3>(p, smem, tmem, keys, from, tab, buf, row, q, ratio, flip, two);
        else expand_tile<N, NG, ZT, 4>(p, smem, tmem, keys, from, tab, buf, row, q, ratio, flip, two);
        wait_st();
        fence_before();
        fence_async();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(keys ? &sh.k_full[buf] : &sh.v_full[buf]);
            mbar_arrive(&sh.ring_empty[st]);
        }
        if (++st == p.depth) st = 0, rpar ^= 1;
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

// The queries of an item's columns. Eight lanes take a column, 16 elements each, where runs of 16 lie in one head and on 16-byte
// boundaries (`vec_q`): stash_queries starts their copies into the buffer of the weights, idle between two
// items, while the partials of the item before are written, and each lane reads back its own. Else a warp takes a column
// and reads it twice.
template <int N, int NG, int ZT>
__device__ __forceinline__ uint32_t stash_at(uint8_t *smem, int i, int warp, int lane) {
    using L = Plan<N, NG, ZT>;
    return smem_u32(smem + L::oP) + ((i * L::kSoft + warp) * 32 + lane) * 32;
}
template <int N, int NG, int ZT>
__device__ __forceinline__ void stash_queries(const TreeParams &p, uint8_t *smem, const Cursor &c, int warp, int lane) {
    using L = Plan<N, NG, ZT>;
    if (NG == 2 || !p.vec_q) return;
    const int rows = p.unit[c.u].nh * p.per, h0 = p.unit[c.u].h0, cols = min(N, c.n * rows - c.c * N);
    const int g0 = p.unit[c.u].gk * kGroup + 16 * (lane & 7);
#pragma unroll 1
    for (int i = 0; i < N / (4 * L::kSoft); ++i) {
        const int col = warp * 4 + (lane >> 3) + i * 4 * L::kSoft;
        const int at = c.c * N + col, node = at / rows, r = at - node * rows, d0 = g0 - (h0 + r / p.per) * p.dk;
        const uint32_t to = stash_at<N, NG, ZT>(smem, i, warp, lane);
        if (col < cols && d0 >= 0 && d0 < p.dk) {
            const __half *from = static_cast<const __half *>(p.t.q) + (int64_t)(c.first + node) * p.t.q_stride_t +
                                 (int64_t)(h0 * p.per + r) * p.t.q_stride_h + d0;
            cp_async16(to, from);
            cp_async16(to + 16, from + 8);
        } else {
            sts128(to, 0, 0, 0, 0);
            sts128(to + 16, 0, 0, 0, 0);
        }
    }
}

__device__ __forceinline__ float power_of_two(int e) {  // -252 .. 254
    return __int_as_float((127 + (e >> 1)) << 23) * __int_as_float((127 + e - (e >> 1)) << 23);
}
// Where the columns keep their own scales their scores are multiplied by 2^(own - wide_base): at most 2^90, and the powers of two
// that leave fp32 belong to columns whose logits are then less than 2^-100 of another's.
__device__ __forceinline__ int wide_base(int top) { return max(kExLow, top - 90); }
// Exponent of the scale at which fp16 holds a column whose largest finite magnitude is `top`: it lies between 2^7 and 2^8 then, and
// a sum of 128 of them below 2^15.
__device__ __forceinline__ int exponent_of(float top) {
    return top > 0.0f ? max(kExLow, min(kExHigh, ((__float_as_int(top) >> 23) & 255) - 127 - 7)) : kNoEx;
}
// A multiple of 2^(kGuard - 24), for which fp16 has kGuard powers of two to spare below: hi and lo terms of it stay what they are
// when they are multiplied by 2^-kGuard or more. It moves a column by 2^-22 of its largest element at most.
constexpr float kGrid = 1.5f * (1 << (kGuard - 1));

// The rotated queries into shared memory (the K-major B operand), each column rounded to fp16 at its own scale, then brought to
// the tile's (or left, `wide`, where the columns are too far apart); returns what takes the scale back out of the logits.
template <int N, int NG, int ZT>
__device__ float rotate_queries(const TreeParams &p, Shared &sh, uint8_t *smem, const Cursor &c, int warp, int lane, bool &wide) {
    using L = Plan<N, NG, ZT>;
    const TreeUnit u = p.unit[c.u];
    const int rows = u.nh * p.per, cols = min(N, c.n * rows - c.c * N);
    const bool fast = NG == 1 && p.vec_q, half = p.t.dtype == CQ_T_F16;
    // coordinates 4 * lane .. of group g of a column's query, placed at its head's elements of the cache row
    auto load = [&](int col, int g, float (&z)[4]) {
        const int at = c.c * N + col, node = at / rows, r = at - node * rows, h = u.h0 + r / p.per;
        const int64_t src = (int64_t)(c.first + node) * p.t.q_stride_t + (int64_t)(u.h0 * p.per + r) * p.t.q_stride_h;
        const int d0 = (u.gk + g) * kGroup + 4 * lane - h * p.dk;
#pragma unroll
        for (int j = 0; j < 4; ++j) z[j] = d0 + j >= 0 && d0 + j < p.dk ? load_q(p, src + d0 + j) : 0.0f;
    };
    // the columns' largest finite magnitudes (what is not finite scales nothing)
    int top = kNoEx, low = -kNoEx;
    if (fast) {
        asm volatile("cp.async.wait_all;\n" ::: "memory");
        const uint32_t inf = half ? 0x7C00u : 0x7F80u;
#pragma unroll 1
        for (int i = 0; i < N / (4 * L::kSoft); ++i) {
            const uint32_t from = stash_at<N, NG, ZT>(smem, i, warp, lane);
            const uint4 v0 = lds128(from), v1 = lds128(from + 16);
            const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
            uint32_t most = 0;  // magnitudes of a 16-bit type are ordered as integers
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t a = w[j] & 0x7FFFu, b = w[j] >> 16 & 0x7FFFu;
                most = max(most, max(a < inf ? a : 0u, b < inf ? b : 0u));
            }
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
            const int ex = exponent_of(half ? __half2float(__ushort_as_half((unsigned short)most)) : __uint_as_float(most << 16));
            if ((lane & 7) == 0) sh.zex[warp * 4 + (lane >> 3) + i * 4 * L::kSoft] = (signed char)ex;
            top = max(top, ex), low = min(low, ex == kNoEx ? -kNoEx : ex);
        }
        top = __reduce_max_sync(0xFFFFFFFFu, top), low = __reduce_min_sync(0xFFFFFFFFu, low);
    } else {
#pragma unroll 1
        for (int col = warp; col < N; col += L::kSoft) {
            float most = 0.0f;
#pragma unroll 1
            for (int g = 0; col < cols && g < u.ngk; ++g) {
                float z[4];
                load(col, g, z);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (fabsf(z[j]) <= 3.4e38f) most = fmaxf(most, fabsf(z[j]));
            }
            const int ex = exponent_of(__uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(most))));
            if (lane == 0) sh.zex[col] = (signed char)ex;
            top = max(top, ex), low = min(low, ex == kNoEx ? -kNoEx : ex);
        }
    }
    if (lane == 0) atomicMax(&sh.ztop, top), atomicMin(&sh.zlow, low);
    bar_sync(1, 32 * L::kSoft);
    top = sh.ztop == kNoEx ? 0 : sh.ztop;
    wide = top - sh.zlow > kGuard;  // not where all columns are zero: 0 - 128
    // a column's own scale, and from there to the tile's
    auto own_of = [&](int col) { return sh.zex[col] == kNoEx ? top : sh.zex[col]; };
    auto down_of = [&](int own) { return __int_as_float((127 - own) << 23); };
    auto shift_of = [&](int own) { return __float2half2_rn(wide ? 1.0f : __int_as_float((127 + own - top) << 23)); };
    auto scaled = [&](__half2 v, __half2 shift) {
        const __half2 x = __hmul2(v, shift);
        return *reinterpret_cast<const uint32_t *>(&x);
    };
    if (fast) {
#pragma unroll 1
        for (int i = 0; i < N / (4 * L::kSoft); ++i) {
            const int sub = lane & 7, col = warp * 4 + (lane >> 3) + i * 4 * L::kSoft;
            const uint32_t from = stash_at<N, NG, ZT>(smem, i, warp, lane);
            const uint4 v0 = lds128(from), v1 = lds128(from + 16);
            const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
            const int own = own_of(col);
            const float down = down_of(own);
            const __half2 shift = shift_of(own);
            F2 z[8];  // elements 2 j and 2 j + 1
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&w[j]));
                const float a = half ? x.x : __uint_as_float(w[j] << 16), b = half ? x.y : __uint_as_float(w[j] & 0xFFFF0000u);
                z[j] = f2_mul(f2(a + b, a - b), f2(down, down));
            }
            const F2 minus = f2(-1.0f, -1.0f);
#pragma unroll
            for (int h = 1; h < 8; h <<= 1)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (!(j & h)) {
                        const F2 x = z[j], y = z[j + h];
                        z[j] = f2_add(x, y), z[j + h] = f2_fma(y, minus, x);
                    }
#pragma unroll 1
            for (int o = 1; o < 8; o <<= 1) {
                const float sign = (sub & o) ? -1.0f : 1.0f;
                const F2 s2 = f2(sign, sign);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float x, y;
                    f2_get(z[j], x, y);
                    z[j] = f2_fma(z[j], s2, f2(__shfl_xor_sync(0xFFFFFFFFu, x, o), __shfl_xor_sync(0xFFFFFFFFu, y, o)));
                }
            }
            uint32_t h2[8];
            const F2 grid = f2(kGrid, kGrid), back = f2(-kGrid, -kGrid);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                z[j] = f2_add(f2_add(z[j], grid), back);
                float x, y;
                f2_get(z[j], x, y);
                h2[j] = scaled(__floats2half2_rn(x, y), shift);
            }
            const uint32_t base = smem_u32(smem + L::oZ) + (sub >> 2) * (N * 128) + (col >> 3) * 1024 + (col & 7) * 128;
            sts128(base + (((2 * (sub & 3)) ^ (col & 7)) << 4), h2[0], h2[1], h2[2], h2[3]);
            sts128(base + (((2 * (sub & 3) + 1) ^ (col & 7)) << 4), h2[4], h2[5], h2[6], h2[7]);
            if (ZT == 2 && half) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float x, y;
                    f2_get(z[j], x, y);
                    const float2 hi = __half22float2(__floats2half2_rn(x, y));
                    h2[j] = scaled(__floats2half2_rn(x - hi.x, y - hi.y), shift);
                }
                sts128(base + L::kZBytes + (((2 * (sub & 3)) ^ (col & 7)) << 4), h2[0], h2[1], h2[2], h2[3]);
                sts128(base + L::kZBytes + (((2 * (sub & 3) + 1) ^ (col & 7)) << 4), h2[4], h2[5], h2[6], h2[7]);
            }
        }
    } else {
#pragma unroll 1
        for (int k = warp * NG; k < N * NG; k += k % NG == NG - 1 ? (L::kSoft - 1) * NG + 1 : 1) {
            const int col = k / NG, g = k % NG;
            float z[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (col < cols && g < u.ngk) load(col, g, z);
            const int own = own_of(col);
            const float down = down_of(own);
            const __half2 shift = shift_of(own);
#pragma unroll
            for (int j = 0; j < 4; ++j) z[j] *= down;
            fwht(z, lane);
#pragma unroll
            for (int j = 0; j < 4; ++j) z[j] = __fadd_rn(__fadd_rn(z[j], kGrid), -kGrid);
            const uint32_t base = smem_u32(smem + L::oZ) + g * L::kZBytes + (col >> 3) * 1024 + (col & 7) * 128;
            auto put = [&](int pos, float x, float y) {
                const __half2 v = __floats2half2_rn(x, y);
                const uint32_t to = base + (pos >> 6) * (N * 128) + ((((pos & 63) >> 3) ^ (col & 7)) << 4) + (pos & 7) * 2;
                sts32(to, scaled(v, shift));
                if (ZT == 2 && half) {
                    const float2 hi = __half22float2(v);
                    sts32(to + NG * L::kZBytes, scaled(__floats2half2_rn(x - hi.x, y - hi.y), shift));
                }
            };
            if (NG == 2 && p.wk == 2) {
                put(position_of(4 * lane, 2), z[0], z[2]);
                put(position_of(4 * lane + 1, 2), z[1], z[3]);
            } else {
                put(4 * lane, z[0], z[1]);
                put(4 * lane + 2, z[2], z[3]);
            }
        }
    }
    return p.k_mult * power_of_two(wide ? wide_base(top) : top);
}

// Who attends drafted token j, as bits over the item's columns.
template <int N>
__device__ void gather_mask(const TreeParams &p, Shared &sh, const Cursor &c, int warp, int warps, int lane) {
    const int rows = p.unit[c.u].nh * p.per, jw = (c.n + 31) / 32;
    for (int k = warp; k < jw * ((N + 31) / 32); k += warps) {
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

__device__ __forceinline__ float warp_max(float x) {  // NaNs count as nothing
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xFFFFFFFF;\n" : "=f"(r) : "f"(x));
    return r;
}

// Scores of X columns for this thread's cache row; with two groups their sum in the ratio r0 : r1 of the row's norms.
template <int N, int NG, int X>
__device__ __forceinline__ void load_scores(uint32_t ts, float (&d)[X], float r0, float r1, bool two) {
    tmem_ld<X>(ts, d);
    wait_ld<X>(d);
    if (NG == 2 && two) {
#pragma unroll
        for (int k = 0; k < X; k += 8) {
            float e[8];
            tmem_ld<8>(ts + N + k, e);
            wait_ld<8>(e);
#pragma unroll
            for (int j = 0; j < 8; ++j) d[k + j] = fmaf(e[j], r1, d[k + j] * r0);
        }
    }
}

// Raises the references of columns cx .. cx + X - 1 whose largest logit of this tile (columns in tensor memory at ts, this
// thread's cache row) passes the weights' range; the factors for what was summed before go to sh.f. All four warps of
// the warpgroup; true if any was raised. Kept out of the loop's straight line: it runs in the first tile and rarely after.
template <int N, int NG, int X>
__device__ __noinline__ bool raise(Shared &sh, uint32_t ts, int cx, float nk, float ln, float r0, float r1, bool two, uint32_t see, int warp, int lane) {
    const int wg = warp >> 2, row = 32 * (warp & 3) + lane;
    float mine = 0.0f;
#pragma unroll 1
    for (int k = 0; k < X; k += 8) {
        float d[8];
        load_scores<N, NG, 8>(ts + k, d, r0, r1, two);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float t = see >> (k + j) & 1 ? fmaf(d[j], nk, ln) : -INFINITY;
            const float x = warp_max(fmaxf(t, -INFINITY));
            if (lane == k + j) mine = x;
        }
    }
    if (lane < X) sh.by_warp[warp][lane] = mine;
    bar_sync(2 + wg, 128);
    bool raised = false;
    if (row < X) {
        const float old = -sh.minus_m[cx + row];
        float x = sh.by_warp[4 * wg][row];
#pragma unroll
        for (int k = 1; k < 4; ++k) x = fmaxf(x, sh.by_warp[4 * wg + k][row]);
        raised = x > old + kRaise;
        sh.f[cx + row] = raised ? ex2(old - x) : 1.0f;
        if (raised) sh.minus_m[cx + row] = -x;
    }
    return bar_or(2 + wg, 128, raised);
}

// The first references of an item's part: the largest finite logits of the tile's first 32 cache rows, by their warp alone. With
// 2^15 above them that holds nearly always, and costs the other warps a barrier.
template <int N, int NG, int X>
__device__ __noinline__ void seed(Shared &sh, uint32_t ts, int cx, float nk, float ln, float r0, float r1, bool two, uint32_t see, int lane) {
    float mine = kNoMax;
#pragma unroll 1
    for (int k = 0; k < X; k += 8) {
        float d[8];
        load_scores<N, NG, 8>(ts + k, d, r0, r1, two);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float t = fmaf(d[j], nk, ln);
            const float x = warp_max((see >> (k + j) & 1) && t < 1e30f ? t : kNoMax);
            if (lane == k + j) mine = x;
        }
    }
    if (lane < X) sh.minus_m[cx + lane] = -fmaxf(mine, kNoMax);
}

// Scales the running sums of columns cx .. cx + X - 1 by the factors of a raise.
__device__ __noinline__ void scale_sums(Shared &sh, uint32_t to, int n, int groups, int cx, int X) {
#pragma unroll 1
    for (int g = 0; g < groups; ++g) {
#pragma unroll 1
        for (int k = 0; k < X; k += 8) {
            float o[8];
            tmem_ld<8>(to + g * n + cx + k, o);
            wait_ld<8>(o);
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] *= sh.f[cx + k + j];
            tmem_st8(to + g * n + cx + k, o);
        }
    }
    wait_st();
}

// Brings the scores of NC columns from c0 on (tensor memory at ts, a warp its own rows) from their own scales to one.
template <int N, int NG, int NC>
__device__ __noinline__ void scale_scores(Shared &sh, uint32_t ts, int c0, bool two) {
    const int base = wide_base(sh.ztop);
#pragma unroll 1
    for (int g = 0; g < (NG == 2 && two ? 2 : 1); ++g) {
#pragma unroll 1
        for (int k = 0; k < NC; k += 8) {
            float d[8];
            tmem_ld<8>(ts + g * N + k, d);
            wait_ld<8>(d);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int ex = sh.zex[c0 + k + j];
                d[j] *= ex == kNoEx ? 1.0f : power_of_two(ex - base);
            }
            tmem_st8(ts + g * N + k, d);
        }
    }
    wait_st();
}

// What a part has summed so far (reference and denominator `old`, the thread's own write) and a chunk's m and x, taken together,
// with the factors for both sums.
__device__ __noinline__ void join_references(float2 old, float &m, float &x, float &before, float &now) {
    const float top = fmaxf(old.x, m);
    before = ex2(old.x - top), now = ex2(m - top);
    x = fmaf(x, now, old.y * before);
    m = top;
}
// Likewise the sums of n columns from c0 on (tensor memory at ts, a thread its own value coordinate).
__device__ __noinline__ void join_sums(Shared &sh, float *out, uint32_t ts, int c0, int n, int wg) {
#pragma unroll 1
    for (int k = 0; k < n; k += 8) {
        float o[8], old[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) old[j] = k + j < n ? out[(size_t)(c0 + k + j) * kGroup] : 0.0f;
        tmem_ld<8>(ts + c0 + k, o);
        wait_ld<8>(o);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (k + j < n) out[(size_t)(c0 + k + j) * kGroup] = fmaf(o[j], sh.f[c0 + k + j], old[j] * sh.by_warp[4 * wg][k + j]);
    }
}

template <int N, int NG, int ZT>
__device__ void softmax_role(const TreeParams &p, Shared &sh, uint8_t *smem, int warp, int lane) {
    using L = Plan<N, NG, ZT>;
    constexpr int NC = N / L::kSoftWG;         // columns of this warpgroup
    constexpr int kSoftThreads = 32 * L::kSoft;
    constexpr int X = NC < 32 ? NC : 32;       // columns per tensor memory load
    const int wg = warp >> 2, q = warp & 3, row = 32 * q + lane, c0 = wg * NC;
    const uint32_t tm = sh.tmem + ((uint32_t)(32 * q) << 16);
    Cursor c = sh.start;
    int i = 0;
    long long place = sh.first;  // of the tile to come
    bool more = true, again = false;  // again: a chunk of the same item's part
    float mult = 0.0f;
    bool wide = false;
    stash_queries<N, NG, ZT>(p, smem, c, warp, lane);
    while (more) {
        // ------------------------------------------ a chunk of an item's part --
        const TreeUnit u = p.unit[c.u];
        const int cols = min(N, c.n * u.nh * p.per - c.c * N), slot = blockIdx.x + c.item;
        if (!again) {
            bar_sync(1, kSoftThreads);  // the item before is finished: the exponents, m, mask may be written
            if (warp == 0 && lane == 0) sh.ztop = kNoEx, sh.zlow = -kNoEx;
            if (row < NC) sh.minus_m[c0 + row] = -kNoMax;
            gather_mask<N>(p, sh, c, warp, L::kSoft, lane);
            bar_sync(1, kSoftThreads);
            mult = rotate_queries<N, NG, ZT>(p, sh, smem, c, warp, lane, wide);
            fence_async();
            fence_before();  // tensor memory reads of the item before
            __syncwarp();
            if (lane == 0 && p.spin == kSpin) mbar_arrive(&sh.z_full);  // a self-test's products wait in vain
            const int i0 = (c.s * p.n_units + c.u) * p.ncol_max + c.c;
            if (c.tile == 0 && warp == 0 && lane == 0)
                p.rec[i0] = make_int2(slot, run_of(sh.total, p.grid, place + c.ntiles - 1) - (int)blockIdx.x + 1);
        }
        const int count = min(kChunk, min(c.ntiles - c.tile, c.left));
        const bool two = NG == 2 && u.ngk == 2;
        F2 l[NC / 2];
#pragma unroll
        for (int k = 0; k < NC / 2; ++k) l[k] = f2(0.0f, 0.0f);
#pragma unroll 1
        for (int it = 0; it < count; ++it, ++i) {
            const int b = i & 1;
            const uint32_t par = (uint32_t)(i >> 1) & 1;
            const int tok = (c.tile + it) * kTile;
            const bool masked = tok + kTile > c.ctx;  // the tile holds drafted tokens
            uint32_t see[(NC + 31) / 32];
#pragma unroll
            for (int k = 0; k < (NC + 31) / 32; ++k) {
                const int j = tok + row - c.ctx;
                see[k] = j >= 0 && j < c.n ? sh.mask[j][(c0 + 32 * k) >> 5] >> (c0 & 31) : 0xFFFFFFFFu;
            }
            wait(p, sh, &sh.sc_full[b], par, 0x47490009u);
            const float nk = sh.scal[b][0][row] * mult, ln = sh.scal[b][1][row], inv = sh.scal[b][2][row];
            float r0 = 1.0f, r1 = 0.0f;
            if (NG == 2) {
                const uint32_t from = smem_u32(smem + L::oRatio) + (b * 2 * kTile + row) * 4;
                r0 = __uint_as_float(lds32(from)), r1 = __uint_as_float(lds32(from + kTile * 4));
            }
            const F2 nk2 = f2(nk, nk), ln2 = f2(ln, ln), inv2 = f2(inv, inv);
            wait(p, sh, &sh.s_full[b], par, 0x4749000Au);
            fence_after();
            if (__builtin_expect(wide, 0)) scale_scores<N, NG, NC>(sh, tm + L::cS + b * NG * N + c0, c0, two);
            // Column by column in halves of X: the denominators of all columns and the logits of one half fit the registers.
#pragma unroll
            for (int hf = 0; hf < NC; hf += X) {
                float d[X];
                const int cx = c0 + hf;
                const uint32_t ts = tm + L::cS + b * NG * N + cx;
                bool raised = false;
                if (__builtin_expect(it == 0, 0)) {
                    if (q == 0) seed<N, NG, X>(sh, ts, cx, nk, ln, r0, r1, two, masked ? see[hf / 32] : 0xFFFFFFFFu, lane);
                    bar_sync(2 + wg, 128);
                }
#pragma unroll 1
                for (int pass = 0;; ++pass) {
                    load_scores<N, NG, X>(ts, d, r0, r1, two);
                    float top = kNoMax;
#pragma unroll
                    for (int k = 0; k < X; k += 4) {  // d = log2 of the weights
                        const float4 m = *reinterpret_cast<const float4 *>(&sh.minus_m[cx + k]);
                        f2_get(f2_add(f2_fma(f2(d[k], d[k + 1]), nk2, ln2), f2(m.x, m.y)), d[k], d[k + 1]);
                        f2_get(f2_add(f2_fma(f2(d[k + 2], d[k + 3]), nk2, ln2), f2(m.z, m.w)), d[k + 2], d[k + 3]);
                    }
                    if (__builtin_expect(masked, 0)) {
#pragma unroll
                        for (int k = 0; k < X; ++k) d[k] = see[hf / 32] >> k & 1 ? d[k] : -INFINITY;
                    }
#pragma unroll
                    for (int k = 0; k < X; k += 2) top = max3(top, d[k], d[k + 1]);
                    if (!bar_or(2 + wg, 128, top > kRaise) || pass) break;
                    raised = raise<N, NG, X>(sh, ts, cx, nk, ln, r0, r1, two, masked ? see[hf / 32] : 0xFFFFFFFFu, warp, lane);
                }
                if (__builtin_expect(raised, 0)) {
#pragma unroll
                    for (int k = 0; k < X; k += 2) {
                        const float2 f = *reinterpret_cast<const float2 *>(&sh.f[cx + k]);
                        l[(hf + k) / 2] = f2_mul(l[(hf + k) / 2], f2(f.x, f.y));
                    }
                    if (it) {  // the first tile's product does not accumulate
                        wait(p, sh, &sh.p_empty, (uint32_t)(i - 1) & 1, 0x4749000Bu);
                        fence_after();
                        scale_sums(sh, tm + L::cO, N, u.ngv, cx, X);
                    }
                }
                if (hf + X == NC) {
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.s_empty[b]);
                }
                if (hf == 0) wait(p, sh, &sh.p_empty, (uint32_t)(i & 1) ^ 1, 0x4749000Cu);
                // weights in fp16: cache row `row`, columns cx .. cx + X - 1 (the MN-major B operand)
                const uint32_t pb = smem_u32(smem + L::oP) + (cx >> 6) * (kTile * 128) + (row >> 3) * 1024 + (row & 7) * 128;
#pragma unroll
                for (int k = 0; k < X; k += 8) {
                    uint32_t h[4];
#pragma unroll
                    for (int j = 0; j < 8; j += 2) {
                        const float x = ex2(d[k + j]), y = ex2(d[k + j + 1]);
                        l[(hf + k + j) / 2] = f2_fma(f2(x, y), inv2, l[(hf + k + j) / 2]);
                        const __half2 v = __floats2half2_rn(x, y);
                        h[j >> 1] = *reinterpret_cast<const uint32_t *>(&v);
                    }
                    sts128(pb + (((((cx + k) & 63) >> 3) ^ (row & 7)) << 4), h[0], h[1], h[2], h[3]);
                }
            }
            fence_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.p_full);
        }
        // ------------------------------------------------ the chunk's partials --
#pragma unroll
        for (int hf = 0; hf < NC; hf += X) {
            float v[X];
#pragma unroll
            for (int k = 0; k < X; k += 2) f2_get(l[(hf + k) / 2], v[k], v[k + 1]);
            // sums over the lanes: each step halves the columns a lane carries, so lane k ends with column k
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                if (o >= X) {
#pragma unroll
                    for (int k = 0; k < X; ++k) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], o);
                } else {
#pragma unroll
                    for (int k = 0; k < o; ++k) {
                        const bool up = lane & o;
                        const float send = up ? v[k] : v[k + o], keep = up ? v[k + o] : v[k];
                        v[k] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, o);
                    }
                }
            }
            if (lane < X) sh.by_warp[warp][hf + lane] = v[0];
        }
        bar_sync(2 + wg, 128);
        if (row < NC && c0 + row < cols) {
            float x = sh.by_warp[4 * wg][row] + sh.by_warp[4 * wg + 1][row] + (sh.by_warp[4 * wg + 2][row] + sh.by_warp[4 * wg + 3][row]);
            float m = -sh.minus_m[c0 + row];
            float2 *ml = &p.ml[(size_t)slot * N + c0 + row];
            if (__builtin_expect(again, 0)) join_references(*ml, m, x, sh.by_warp[4 * wg][row], sh.f[c0 + row]);
            *ml = make_float2(m, x);
        }
        place += count;
        c.left -= count;
        c.tile += count;
        more = c.left > 0;
        const bool merge = again;
        again = more && c.tile < c.ntiles;
        if (merge || again) bar_sync(2 + wg, 128);  // the factors; the references may be written again
        if (more && !again) {
            place += item_cost(N);
            c.next_item(p, N);
        }
        wait(p, sh, &sh.p_empty, (uint32_t)(i - 1) & 1, 0x4749000Du);
        fence_after();
        if (more && !again) stash_queries<N, NG, ZT>(p, smem, c, warp, lane);
        const int nat = NG == 2 ? natural_of(row, p.wv) : row;
        for (int g = 0; g < u.ngv; ++g) {
            float *out = p.part + ((size_t)slot * NG + g) * N * kGroup + nat;
            if (__builtin_expect(merge, 0)) {
                join_sums(sh, out, tm + L::cO + g * N, c0, min(NC, cols - c0), wg);
                continue;
            }
#pragma unroll 1
            for (int k = 0; k < NC; k += 8) {
                if (c0 + k >= cols) break;
                float o[8];
                tmem_ld<8>(tm + L::cO + g * N + c0 + k, o);
                wait_ld<8>(o);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c0 + k + j < cols) out[(size_t)(c0 + k + j) * kGroup] = o[j];
            }
        }
    }
}

template <int N, int NG, int ZT>
__global__ void __launch_bounds__(Plan<N, NG, ZT>::kThreads, 1) tree_kernel(const __grid_constant__ TreeParams p) {
    using L = Plan<N, NG, ZT>;
    extern __shared__ __align__(1024) uint8_t smem[];
    constexpr int kIssuer = L::kSoft + L::kExp;
    Shared &sh = *reinterpret_cast<Shared *>(smem + L::oShared);
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    if (smem_u32(smem) != kSmemFirst) {  // the tables' addresses count on it; the host has checked (smem_check)
        if (tid == 0) atomicOr(p.status, 0x47490010u);
        return;
    }
    if (tid == 0) {
        sh.abort = 0;
        sh.bad = 0;
#pragma unroll 1
        for (int i = 0; i < p.depth; ++i) {
            mbar_init(&sh.ring_full[i], 128);
            mbar_init(&sh.ring_empty[i], 8);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.k_full[i], 4);
            mbar_init(&sh.k_empty[i], 1);
            mbar_init(&sh.v_full[i], 4);
            mbar_init(&sh.v_empty[i], 1);
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.s_empty[i], L::kSoft);
            mbar_init(&sh.sc_full[i], 8);
        }
        mbar_init(&sh.p_full, L::kSoft);
        mbar_init(&sh.p_empty, 1);
        mbar_init(&sh.z_full, L::kSoft);
        mbar_init(&sh.drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (NG == 1) {
        fill_table(p.tab_k, p.tk, p.wk, p.wk == 2 && wide_two(N));
        if (p.tab_v != p.tab_k) fill_table(p.tab_v, p.tv, p.wv, p.wv == 2 && wide_two(N));
    }
    __syncthreads();
    const bool work = find_run<N, L::kThreads>(p, sh);  // uniform
    if (blockIdx.x == 0 && tid == 0 && sh.bad) atomicOr(p.status, kStatusIndex);
    if (!work) return;
    if (warp == kIssuer) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(&sh.tmem)), "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::);
    }
    fence_before();
    __syncthreads();
    fence_after();
    // A softmax thread of many columns keeps logits and denominators in registers: the others give theirs up.
    if (warp < L::kSoft) {
        if (L::kSoftWG == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(L::kSoftRegs));
        softmax_role<N, NG, ZT>(p, sh, smem, warp, lane);
    } else if (warp < L::kSoft + L::kExp) {
        if (L::kSoftWG == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(L::kExpRegs));
        const int row = 32 * (warp & 3) + lane;
        expand_role<N, NG, ZT>(p, sh, smem, warp < L::kSoft + 4, row, warp & 3, lane);
    } else {
        if (L::kSoftWG == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(L::kRestRegs));
        if (warp == kIssuer) issue_role<N, NG, ZT>(p, sh, smem);
        else if (warp < kIssuer + 3) fetch_role<N, NG, ZT>(p, sh, smem, tid - 32 * (kIssuer + 1));
    }
    fence_before();
    __syncthreads();
    if (warp == kIssuer) {
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
    asm volatile("griddepcontrol.wait;\n" ::: "memory");  // every block: what follows this kernel also follows the one before it
    if (first >= cols) return;
    int2 rec = p.rec[item];
    if (rec.x < 0 || rec.y < 0 || rec.x > p.slots - rec.y) rec.y = 0;  // an item that no block wrote
    const bool many = rec.y > kFewParts;
    for (int k = many ? 0 : warp; k < CG && first + k < cols; k += many ? 1 : kJoinWarps) {
        const int col = first + k;
        float M = kNoMax, sum = 0.0f, acc[NG][4];
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[g][j] = 0.0f;
        // weighted sums in part order, rescaled where a part has a larger reference: all loads are independent
#pragma unroll 2
        for (int a = many ? warp : 0; a < rec.y; a += many ? kJoinWarps : 1) {
            const float2 ml = p.ml[(size_t)(rec.x + a) * N + col];
            float4 v[NG];
#pragma unroll
            for (int g = 0; g < NG; ++g)
                if (g < u.ngv) v[g] = *reinterpret_cast<const float4 *>(p.part + (((size_t)(rec.x + a) * NG + g) * N + col) * kGroup + 4 * lane);
            const float top = fmaxf(M, ml.x), f = ex2(M - top), w = ex2(ml.x - top);
            M = top;
            sum = fmaf(ml.y, w, sum * f);
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                if (g >= u.ngv) break;
                acc[g][0] = fmaf(v[g].x, w, acc[g][0] * f), acc[g][1] = fmaf(v[g].y, w, acc[g][1] * f);
                acc[g][2] = fmaf(v[g].z, w, acc[g][2] * f), acc[g][3] = fmaf(v[g].w, w, acc[g][3] * f);
            }
        }
        if (many) {  // uniform in the block: the warps' sums meet in warp 0
            __syncthreads();
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int j = 0; j < 4; ++j) s_acc[warp][g][4 * lane + j] = acc[g][j];
            if (lane == 0) s_ml[warp] = make_float2(M, sum);
            __syncthreads();
            if (warp) continue;
            float top = kNoMax;
            for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, s_ml[w].x);
            sum = 0.0f;
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[g][j] = 0.0f;
            for (int w = 0; w < kJoinWarps; ++w) {
                const float f = ex2(s_ml[w].x - top);
                sum = fmaf(s_ml[w].y, f, sum);
#pragma unroll
                for (int g = 0; g < NG; ++g)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[g][j] = fmaf(s_acc[w][g][4 * lane + j], f, acc[g][j]);
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
// Level tables at the top, the larger one first; the ring has what is left behind the fixed part. Its stages, or 0 where fewer
// than two fit.
template <int N, int NG, int ZT>
int lay_out(int wk, int wv, bool same, uint32_t &tab_k, uint32_t &tab_v) {
    int end = kSmemLast;
    tab_k = tab_v = 0;
    if (NG == 1) {
        auto place = [&](int w, int top) { return top - table_bytes(w, N) & -table_bytes(w, N); };
        const bool k_first = table_bytes(wk, N) >= table_bytes(wv, N);
        const int a = place(k_first ? wk : wv, kTabTop), b = same ? a : place(k_first ? wv : wk, a);
        tab_k = k_first ? a : b;
        tab_v = k_first ? b : a;
        end = b;
    }
    const int depth = std::min(kMaxDepth, (end - kSmemFirst - Plan<N, NG, ZT>::oRing) / Stage<NG>::bytes(wk, wv));
    return depth >= 2 ? depth : 0;
}

// Two four-bit tables leave 64 columns two stages (and 128 columns one: shape_of then takes 64).
static_assert((kTabTop - 2 * table_bytes(4, 64) - kSmemFirst - Plan<64, 1, 2>::oRing) / Stage<1>::bytes(4, 4) >= 2, "stages");
static_assert(Plan<128, 1, 2>::oRing == Plan<128, 1, 1>::oRing, "one layout for both kernels of 128 columns");
static_assert((kSmemLast - kSmemFirst - Plan<64, 2, 2>::oRing) / Stage<2>::bytes(4, 4) >= 2, "stages");

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
    // 128 columns leave room for one large level table, or for two where a stage of codes is small
    const bool same = g.k_bits == g.v_bits && std::equal(g.k_codebook, g.k_codebook + levels_of(g.k_bits), g.v_codebook);
    uint32_t tk, tv;
    if (s.N == 128 && !lay_out<128, 1, 1>(width_of(g.k_bits), width_of(g.v_bits), same, tk, tv)) s.N = 64;
    s.ncol_max = std::max(1, (most + s.N - 1) / s.N);
    s.items = (size_t)n_seqs * s.n_units * s.ncol_max;
    s.slots = s.items + sm_count();
    return s;
}

size_t up16(size_t n) { return (n + 15) / 16 * 16; }

// What rounding x to fp16 leaves, for normal fp16 values: ties to even, by the bits.
float round_f16(float x) {
    uint32_t u;
    std::memcpy(&u, &x, 4);
    u = (u + 0xFFFu + (u >> 13 & 1)) & ~0x1FFFu;
    std::memcpy(&x, &u, 4);
    return x;
}

// Level tables as bytes. The levels are scaled so that the largest lies in [1, 4) and fp16 holds them well: of 4096 scales the
// one with the least sum of squared errors, after the part that all levels share is taken out again with the
// scale (eight magnitudes are then off by 2^-15 or so instead of 2^-12; with 256 scales half as well). Returns what takes the scale out.
// The search is a pure function of the levels; a thread keeps its last results, by content.
float byte_table(const float *lv, uint32_t *t) {
    struct Found {
        float lv[16];
        uint32_t t[8];
        float back;
    };
    static thread_local Found found[4];
    static thread_local int filled = 0, next = 0;
    for (int i = 0; i < filled; ++i)
        if (std::equal(lv, lv + 16, found[i].lv)) {
            std::copy(found[i].t, found[i].t + 8, t);
            return found[i].back;
        }
    Found f;
    std::copy(lv, lv + 16, f.lv);
    float mag[16], top = 0.0f;  // the distinct magnitudes
    int n = 0;
    for (int i = 0; i < 16; ++i) {
        const float m = std::fabs(lv[i]);
        top = std::max(top, m);
        if (m != 0.0f && std::find(mag, mag + n, m) == mag + n) mag[n++] = m;
    }
    int e = 0;
    if (top > 0.0f) std::frexp(top, &e), --e;
    double best = 1e300, scale = std::ldexp(1.0, -e), back = 1.0 / scale;
    double xx = 0.0;
    for (int i = 0; i < n; ++i) xx += (double)mag[i] * mag[i];
    for (int k = 0; k < 4096 && n; ++k) {
        const double s = std::ldexp(1.0 + k / 4096.0, -e);
        double xh = 0.0, hh = 0.0;
        for (int i = 0; i < n; ++i) {
            const float h = round_f16((float)(mag[i] * s));
            xh += (double)mag[i] * h, hh += (double)h * h;
        }
        const double left = xx - xh * xh / hh;  // the least sum of (mag - factor * h)^2
        if (left < best) best = left, scale = s, back = xh / hh;
    }
    for (int i = 0; i < 8; ++i) f.t[i] = 0;
    for (int i = 0; i < 16; ++i) {
        const uint32_t b = __half_as_ushort(__float2half_rn((float)(lv[i] * scale)));
        f.t[i / 4] |= (b & 255u) << (8 * (i & 3));
        f.t[4 + i / 4] |= (b >> 8) << (8 * (i & 3));
    }
    f.back = (float)back;
    found[next] = f;
    next = (next + 1) % 4;
    filled = std::min(filled + 1, 4);
    std::copy(f.t, f.t + 8, t);
    return f.back;
}

// Bytes at the start of a block's shared memory that the system keeps on the current device (cached per device), or -1.
int reserved_smem() {
    static std::atomic<int> cache[64];  // one more than the bytes
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        cudaGetLastError();
        return -1;
    }
    int n = cache[dev].load(std::memory_order_relaxed);
    if (!n) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrReservedSharedMemoryPerBlock, dev) != cudaSuccess) {
            cudaGetLastError();
            return -1;
        }
        cache[dev].store(++n, std::memory_order_relaxed);  // every writer stores the same value
    }
    return n - 1;
}

template <int N, int NG, int ZT>
int launch_main(TreeParams &p, cudaStream_t st) {
    p.stage = Stage<NG>::bytes(p.wk, p.wv);
    p.depth = lay_out<N, NG, ZT>(p.wk, p.wv, p.wk == p.wv && std::equal(p.tk, p.tk + 8, p.tv), p.tab_k, p.tab_v);
    if (!p.depth) return set_error(CQ_ERR_SHAPE, "no room for the level tables");
    int rc = tree_smem_check(reserved_smem());
    if (rc) return rc;
    rc = ensure_smem(reinterpret_cast<const void *>(tree_kernel<N, NG, ZT>), kSmemLast - kSmemFirst);
    if (rc) return rc;
    tree_kernel<N, NG, ZT><<<p.grid, Plan<N, NG, ZT>::kThreads, kSmemLast - kSmemFirst, st>>>(p);
    return CQ_OK;
}

}  // namespace

int tree_smem_check(int reserved) {
    if (reserved == kSmemFirst) return CQ_OK;
    return set_error(CQ_ERR_CUDA, "tree attention counts on shared memory from byte %d on, and the system keeps %d bytes", kSmemFirst, reserved);
}

size_t tree_workspace(const cq_kv_geom &g, int n_seqs, int max_nodes) {
    if (!n_seqs || !max_nodes) return 0;
    TreeUnit u[kMaxUnits];
    const Shape s = shape_of(g, n_seqs, max_nodes, u);
    return up16(s.items * sizeof(int2)) + up16(s.slots * s.N * sizeof(float2)) + s.slots * s.ng * s.N * kGroup * sizeof(float);
}

int launch_kv_tree_attend(const cq_kv_geom &g, const cq_kv_tree &t, const float *lk, const float *lv, bool give_up, void *stream) {
    TreeParams p;
    const Shape s = shape_of(g, t.n_seqs, t.max_nodes, p.unit);
    if (s.slots > (size_t)INT_MAX / 2 || (s.N + 7) / 8 > 65535)
        return set_error(CQ_ERR_SHAPE, "%d requests of up to %d drafted tokens are too many for one call", t.n_seqs, t.max_nodes);
    p.t = t;
    p.n_units = s.n_units;
    p.hq = g.n_q_heads, p.per = g.n_q_heads / g.n_kv_heads, p.dk = g.head_dim_k, p.dv = g.head_dim_v;
    p.wk = width_of(g.k_bits), p.wv = width_of(g.v_bits);
    p.kgroups = in_padded(g.n_kv_heads * p.dk) / kGroup, p.vgroups = in_padded(g.n_kv_heads * p.dv) / kGroup;
    p.vec_q = p.dk % 16 == 0 && (reinterpret_cast<uintptr_t>(t.q) & 15) == 0 && t.q_stride_t % 8 == 0 && t.q_stride_h % 8 == 0;
    // t / block_size for t < 2^31: a product with 2^(31 + l) / block_size rounded up, 2^l >= block_size
    int l = 0;
    while (l < 31 && (1u << l) < (unsigned)t.block_size) ++l;
    p.div_shift = 31 + l;
    p.div_mul = (uint32_t)(((1ull << (31 + l)) + (unsigned)t.block_size - 1) / (unsigned)t.block_size);
    if (!t.max_blocks) p.t.block_table = t.cu_nodes, p.t.table_stride = 0;  // no token is read, but entry 0 is
    p.slots = (int)s.slots;
    p.spin = give_up ? 4 : kSpin;
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
        case 16: rc = launch_main<16, 1, 2>(p, st); break;
        case 32: rc = launch_main<32, 1, 2>(p, st); break;
        case 64: rc = launch_main<64, 1, 2>(p, st); break;
        default: rc = t.dtype == CQ_T_F16 ? launch_main<128, 1, 2>(p, st) : launch_main<128, 1, 1>(p, st); break;
        }
    } else {
        rc = s.N == 16 ? launch_main<16, 2, 2>(p, st) : launch_main<64, 2, 2>(p, st);
    }
    if (rc) return rc;
    // A block per column where they are few (its warps share long rows of parts), a warp per column otherwise: one for each while
    // that is a few blocks per SM, four columns after another beyond (a block is mostly latency: 36 against 26 us for 65536).
    const size_t columns = s.items * s.N;
    const int cg = columns <= 4 * (size_t)p.grid ? 1 : columns <= 128 * (size_t)p.grid ? 8 : std::min(s.N, 32);
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
