// cq_plan.cu -- block tables and slot maps of a step, from the requests' lengths.
//
// Two prefix sums over the requests (new tokens, and blocks taken from the
// free stack) fix every output; everything else is local. The step is
// latency: a few hundred KB at most, so one launch does it without any
// communication between blocks. Each block scans the lengths itself (12 bytes a
// request, from L2), a tile of kTile requests at a time in shared memory, and
// then writes its own equal share of the tokens, each of which finds its
// request by a binary search of the tile's prefix sums. A token's block comes from
// the table row if it was held before the step, else straight from the free
// stack, so no token waits for the table entries that other warps write.
//
// Bound by latency: 33 requests with 0 to 32 new tokens each take 7 to 8 us from cold caches, 1021 with up to 300
// (1.9 MB) 8 to 9, in steps of 12 to 16 us that are the call's own host time.
#include <cuda_runtime.h>

#include <algorithm>

#include "cq_paged.h"

namespace cq {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 4;                  // requests per thread and tile
constexpr int kTile = kThreads * kPer;

struct PlanParams {
    cq_kv_step s;
    unsigned int *status;
    int per;  // tokens per block
};

struct Two {
    int a, b;
};
// Sums of lengths and blocks, held at 2^31 - 1: past that no token has a place, and the order of adding does not matter.
__device__ __forceinline__ int held_sum(int x, int y) { return (int)min((unsigned)x + (unsigned)y, 0x7FFFFFFFu); }
__device__ __forceinline__ Two operator+(Two x, Two y) { return {held_sum(x.a, y.a), held_sum(x.b, y.b)}; }

__global__ void __launch_bounds__(kThreads) kv_plan_kernel(const __grid_constant__ PlanParams p) {
    __shared__ int s_cu[kTile + 1], s_dem[kTile], s_len[kTile], s_held[kTile], s_extra[kTile];
    __shared__ Two s_warp[kThreads / 32];
    const cq_kv_step &S = p.s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int bs = S.block_size, n_free = S.n_free[0];
    const long long t0 = (long long)blockIdx.x * p.per, t1 = min((long long)S.n_tokens, t0 + p.per);
    Two carry{0, 0};
    bool bad = false;
    for (int base = 0; base < S.n_seqs; base += kTile) {
        const int n = min(kTile, S.n_seqs - base);
        Two mine[kPer], sum{0, 0};
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int j = tid * kPer + i;
            mine[i] = Two{0, 0};
            if (j < n) {
                const int len = max(S.seq_lens[base + j], 0), add = max(S.new_lens[base + j], 0);
                const int held = min(max(S.held[base + j], 0), S.max_blocks);
                long long need = add ? ((long long)len + add + bs - 1) / bs : 0;
                if (need > S.max_blocks) need = S.max_blocks, bad = true;
                mine[i] = Two{add, max((int)need - held, 0)};
                s_len[j] = len;
                s_held[j] = held;
                s_extra[j] = mine[i].b;
            }
            sum = sum + mine[i];
        }
        Two inc = sum;  // inclusive scan over the warp, then over the warps
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const Two up{__shfl_up_sync(0xFFFFFFFFu, inc.a, o), __shfl_up_sync(0xFFFFFFFFu, inc.b, o)};
            if (lane >= o) inc = inc + up;
        }
        if (lane == 31) s_warp[warp] = inc;
        __syncthreads();
        Two before = carry, total = carry;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) before = before + s_warp[w];
            total = total + s_warp[w];
        }
        Two run{__shfl_up_sync(0xFFFFFFFFu, inc.a, 1), __shfl_up_sync(0xFFFFFFFFu, inc.b, 1)};
        run = lane ? before + run : before;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int j = tid * kPer + i;
            if (j < n) {
                s_cu[j] = run.a;
                s_dem[j] = run.b;
                // outputs by request: each block writes the tiles of its turn
                if ((base / kTile) % gridDim.x == blockIdx.x) {
                    S.cu_new[base + j] = run.a;
                    S.held_out[base + j] = s_held[j] + mine[i].b;
                }
            }
            run = run + mine[i];
        }
        if (tid == 0) s_cu[n] = total.a;
        __syncthreads();
        // the tokens of this tile that are this block's
        const long long a = max(t0, (long long)carry.a), b = min(t1, (long long)total.a);
        for (long long t = a + tid; t < b; t += kThreads) {
            int lo = 0, hi = n - 1;  // last request that starts at or before t (empty ones share their start)
            while (lo < hi) {
                const int m = (lo + hi + 1) >> 1;
                if (s_cu[m] <= t) lo = m;
                else hi = m - 1;
            }
            const long long pos = (long long)s_len[lo] + (t - s_cu[lo]);
            const long long blk = pos / bs;
            int block = -1;
            if (pos > 0x7FFFFFFF) {
                // no position, and no slot
            } else if (blk < s_held[lo]) {
                block = S.block_table[(base + lo) * S.table_stride + blk];
            } else if (blk < S.max_blocks) {
                const long long at = (long long)n_free - 1 - s_dem[lo] - (blk - s_held[lo]);
                if (at >= 0 && at < S.free_cap) block = S.free_list[at];
            }
            const long long slot = block < 0 ? -1 : (long long)block * bs + (pos - blk * bs);
            if (slot < 0 || slot > 0x7FFFFFFF) bad = true;
            S.slots[t] = slot > 0x7FFFFFFF ? -1 : (int)slot;
            S.positions[t] = pos > 0x7FFFFFFF ? -1 : (int)pos;
            S.token_seq[t] = base + lo;
        }
        // the table entries of the blocks taken, a warp per request
        for (int j = blockIdx.x * (kThreads / 32) + warp; j < n; j += gridDim.x * (kThreads / 32)) {
            const int extra = s_extra[j], held = s_held[j];
            for (int i = lane; i < extra; i += 32) {
                const long long at = (long long)n_free - 1 - s_dem[j] - i;
                const bool have = at >= 0 && at < S.free_cap;
                S.block_table[(base + j) * S.table_stride + held + i] = have ? S.free_list[at] : -1;
                bad |= !have;
            }
        }
        carry = total;
        __syncthreads();
    }
    for (long long t = max(t0, (long long)carry.a) + tid; t < t1; t += kThreads) {
        S.slots[t] = -1;
        S.positions[t] = -1;
        S.token_seq[t] = -1;
    }
    if (blockIdx.x == 0 && tid == 0) {
        S.cu_new[S.n_seqs] = carry.a;
        S.n_free_out[0] = (int)max((long long)n_free - carry.b, -0x80000000ll);
        bad |= carry.a > S.n_tokens;
    }
    if (bad) atomicOr(p.status, kStatusIndex);
}

}  // namespace

int launch_kv_plan(const cq_kv_step &s, void *stream) {
    PlanParams p;
    p.s = s;
    p.status = device_status_ptr();
    if (!p.status) return set_error(CQ_ERR_CUDA, "no device status word");
    // a token is a search and three stores: two tokens a thread, at most two blocks an SM
    const int grid = (int)std::max(1ll, std::min(2ll * sm_count(), ((long long)s.n_tokens + 2 * kThreads - 1) / (2 * kThreads)));
    p.per = (int)(((long long)s.n_tokens + grid - 1) / grid);
    kv_plan_kernel<<<grid, kThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return set_error(CQ_ERR_CUDA, "plan launch: %s", cudaGetErrorString(e));
    return CQ_OK;
}

}  // namespace cq
