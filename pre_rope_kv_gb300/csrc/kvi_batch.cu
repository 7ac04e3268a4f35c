// kvi_batch.cu -- block tables, slots and positions of a step's rows, from the
// requests' lengths (kvi_batch_tables).
//
// Request r holds ctx keys and asks for n more rows.  With had = ceil(ctx / B) and
// has = ceil((ctx + n) / B) it needs has - had blocks; prefix sums over the
// requests say which free blocks they are, where its rows begin and, of finished
// requests, where their blocks go in the ring.  A row's slot then is
// block(position / B) * B + position % B, with the block from the table (the
// request's last one, partly filled) or from the ring (a new one).
//
// A launch has as many blocks as rows want, and each scans the lengths of all
// requests by itself (32 KB at most, from L2): no block waits for another, and a
// step is one launch without a workspace.  What bounds it is that chain of
// latencies (lengths, scan, search, a block's number, a store): 64 requests of one
// token 3.7 us, 16 prompts of 3 thousand rows 3.4 us, 1000 requests of 71 thousand
// rows 6.9 us.
#include <cuda_runtime.h>

#include <algorithm>

#include "kvi_attn.cuh"

namespace kvi {

namespace {

struct BatchParams {
    int32_t R;
    const int32_t *ctx_lens, *new_lens;
    int32_t *tables;
    int32_t max_blocks, num_blocks, B, shared;
    int32_t *free_ids;
    const int64_t *free_at;
    int64_t *free_at_out;
    int32_t *ctx_out, *q_start;
    int32_t total_rows;
    int32_t *positions;
    int64_t *slots;
    int32_t *status;
};

// Exclusive sums over the block's threads, and the sums of all, of three numbers
// (64 bits: what is asked for may be far more than there is).
struct Three {
    int64_t blocks, rows, back;
};
template <int WARPS>
__device__ __forceinline__ Three block_scan(const Three &a, Three *s_warp, Three &all)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Three sum = a;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, sum.blocks, o), y = __shfl_up_sync(0xffffffffu, sum.rows, o),
                      z = __shfl_up_sync(0xffffffffu, sum.back, o);
        if (lane >= o) {
            sum.blocks += x;
            sum.rows += y;
            sum.back += z;
        }
    }
    if (lane == 31) s_warp[warp] = sum;
    __syncthreads();
    all = Three{0, 0, 0};
    Three before{sum.blocks - a.blocks, sum.rows - a.rows, sum.back - a.back};
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        const Three v = s_warp[w];
        if (w < warp) {
            before.blocks += v.blocks;
            before.rows += v.rows;
            before.back += v.back;
        }
        all.blocks += v.blocks;
        all.rows += v.rows;
        all.back += v.back;
    }
    __syncthreads();
    return before;
}

// The last i in [0, n) with at[i] <= x (at[0] <= x, never decreasing)
__device__ __forceinline__ int last_at_most(const int32_t *at, int n, int32_t x)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (at[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// What a request asks for, by its own numbers alone (n < 0: it has finished).
struct Ask {
    int32_t rows;       // 0 of a bad request
    int32_t had, need;  // blocks it has and needs
    int32_t back;       // blocks that go back to the ring
    int error;
};
__device__ __forceinline__ Ask ask_of(const BatchParams &p, int32_t ctx, int32_t n)
{
    const int64_t room = min((int64_t)p.max_blocks * p.B, (int64_t)INT32_MAX), end = (int64_t)ctx + max(n, 0);
    Ask a{0, 0, 0, 0, KVI_OK};
    if (ctx < 0 || ctx > room || (n > 0 && ctx < p.shared)) a.error = KVI_ERR_OUT_OF_RANGE;
    else if (end > room) a.error = KVI_ERR_CAPACITY;
    if (a.error) return a;
    const uint32_t B = (uint32_t)p.B, less = B - 1;
    a.had = (int32_t)(((uint32_t)ctx + less) / B);
    a.rows = max(n, 0);
    if (n > 0) a.need = (int32_t)(((uint32_t)end + less) / B) - a.had;
    if (n < 0) a.back = max(0, a.had - (int32_t)((uint32_t)p.shared / B));
    return a;
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS) batch_kernel(const __grid_constant__ BatchParams p)
{
    extern __shared__ int32_t s_all[];
    int32_t *s_start = s_all, *s_back = s_start + p.R + 1, *s_ctx = s_back + p.R + 1, *s_need = s_ctx + p.R;
    int32_t *s_new = s_need;  // (until the request's turn comes)
    constexpr int kWarps = THREADS / 32;
    __shared__ Three s_warp[kWarps];
    const int tid = threadIdx.x;
    const bool first = blockIdx.x == 0;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t head = p.free_at[0], tail = p.free_at[1];
#pragma unroll 4
    for (int r = tid; r < p.R; r += THREADS) {
        s_ctx[r] = p.ctx_lens[r];
        s_new[r] = p.new_lens[r];
    }
    const bool ring = head >= 0 && tail >= head && tail - head <= p.num_blocks;
    const int64_t avail = ring ? tail - head : 0;
    if (!ring && first && tid == 0) record_status(p.status, KVI_ERR_OUT_OF_RANGE);
    __syncthreads();

    // ---- what is asked for, in the requests' order
    const int per = (p.R + THREADS - 1) / THREADS, r0 = min(p.R, tid * per), r1 = min(p.R, r0 + per);
    Three asked{0, 0, 0}, all;
    for (int r = r0; r < r1; ++r) {
        const Ask a = ask_of(p, s_ctx[r], s_new[r]);
        if (a.error && first) record_status(p.status, a.error);
        asked.blocks += a.need;
        asked.rows += a.rows;
        asked.back += a.back;
    }
    Three at = block_scan<kWarps>(asked, s_warp, all);
    const bool returns = ring && all.back <= p.num_blocks - avail;
    if (!returns && ring && first && tid == 0) record_status(p.status, KVI_ERR_CAPACITY);

    // ---- what is granted: in order while blocks and rows last
    int64_t begin = at.rows, all_rows = all.rows, all_taken = all.blocks;
    if (all.blocks > avail || all.rows > p.total_rows) {
        Three granted{0, 0, 0}, sum;
        int64_t blocks = at.blocks, rows = at.rows;
        for (int r = r0; r < r1; ++r) {
            const Ask a = ask_of(p, s_ctx[r], s_new[r]);
            blocks += a.need;
            rows += a.rows;
            if (a.rows > 0 && (a.need == 0 || blocks <= avail) && rows <= p.total_rows) {
                granted.blocks += a.need;
                granted.rows += a.rows;
            } else if (a.rows > 0 && first) {
                record_status(p.status, KVI_ERR_CAPACITY);
            }
        }
        begin = block_scan<kWarps>(granted, s_warp, sum).rows;
        all_rows = sum.rows;
        all_taken = sum.blocks;
    }
    for (int r = r0; r < r1; ++r) {
        const int32_t ctx = s_ctx[r], n = s_new[r];
        const Ask a = ask_of(p, ctx, n);
        at.rows += a.rows;
        const bool got = a.rows > 0 && (a.need == 0 || at.blocks + a.need <= avail) && at.rows <= p.total_rows;
        s_start[r] = (int32_t)begin;
        s_back[r] = (int32_t)min(at.back, (int64_t)INT32_MAX);
        s_need[r] = got ? (int32_t)at.blocks : 0;
        if (first) {
            p.q_start[r] = (int32_t)begin;
            p.ctx_out[r] = n < 0 && !a.error && returns ? 0 : got ? ctx + n : ctx;
        }
        if (got) begin += a.rows;
        at.blocks += a.need;
        at.back += a.back;
    }
    if (tid == 0) {
        s_start[p.R] = (int32_t)all_rows;
        s_back[p.R] = returns ? (int32_t)all.back : 0;
        if (first) {
            p.q_start[p.R] = (int32_t)all_rows;
            p.free_at_out[0] = head + (ring ? all_taken : 0);
            p.free_at_out[1] = tail + (returns ? all.back : 0);
        }
    }
    __syncthreads();

    // ---- rows: slots and positions, and the tables' new entries
    const int32_t real = s_start[p.R], head_in = ring ? (int32_t)(head % p.num_blocks) : 0;
    const int64_t stride = (int64_t)gridDim.x * THREADS;
#pragma unroll 2
    for (int64_t row = (int64_t)blockIdx.x * THREADS + tid; row < p.total_rows; row += stride) {
        int32_t pos = 0;
        int64_t slot = -1;
        if (row < real) {
            const int r = last_at_most(s_start, p.R, (int32_t)row);
            const int32_t ctx = s_ctx[r];
            pos = ctx + ((int32_t)row - s_start[r]);
            const int32_t col = (int32_t)((uint32_t)pos / (uint32_t)p.B), off = pos - col * p.B;
            const int32_t had = (int32_t)(((uint32_t)ctx + (uint32_t)(p.B - 1)) / (uint32_t)p.B);
            int32_t *entry = p.tables + (int64_t)r * p.max_blocks + col;
            int32_t id;
            if (col >= had) {
                int64_t i = (int64_t)head_in + s_need[r] + (col - had);
                if (i >= p.num_blocks) i -= p.num_blocks;
                id = p.free_ids[i];
                if (off == 0) *entry = id;
            } else {
                id = *entry;
            }
            if ((uint32_t)id < (uint32_t)p.num_blocks)
                slot = (int64_t)id * p.B + off;
            else
                record_status(p.status, KVI_ERR_OUT_OF_RANGE);
        }
        p.positions[row] = pos;
        p.slots[row] = slot;
    }
    // ---- finished requests' blocks (from the last thread on: the first have rows)
    const int32_t returned = s_back[p.R], tail_in = ring ? (int32_t)(tail % p.num_blocks) : 0;
    for (int64_t i = stride - 1 - ((int64_t)blockIdx.x * THREADS + tid); i < returned; i += stride) {
        const int r = last_at_most(s_back, p.R, (int32_t)i);
        int64_t to = (int64_t)tail_in + i;
        if (to >= p.num_blocks) to -= p.num_blocks;
        p.free_ids[to] = p.tables[(int64_t)r * p.max_blocks + p.shared / p.B + ((int32_t)i - s_back[r])];
    }
}

// A row and thread while an SM has one block.  A thread scans R / THREADS requests:
// 512 threads for many requests, 256 for few, whose warps' sums are fewer (us, 256
// and 512 threads: 64 requests 3.6, 4.1; 1000 requests, 71 thousand rows, 8.0, 6.9).
template <int THREADS>
cudaError_t run_batch(const BatchParams &p, cudaStream_t s)
{
    const cudaError_t e = smem_opt_in(batch_kernel<THREADS>, (4 * KVI_MAX_REQUESTS + 2) * 4);
    if (e != cudaSuccess) return e;
    const int64_t wanted = std::max<int64_t>(((int64_t)p.total_rows + THREADS - 1) / THREADS, p.R / 32);
    return launch_chained(batch_kernel<THREADS>, dim3((unsigned)std::min<int64_t>(std::max<int64_t>(wanted, 1), kPlanSms)), THREADS,
                          (4 * p.R + 2) * 4, s, p);
}

}  // namespace

}  // namespace kvi

using namespace kvi;

extern "C" kvi_status kvi_batch_tables(int32_t R, const int32_t *d_ctx_lens, const int32_t *d_new_lens,
                                       int32_t *d_block_tables, int32_t max_blocks, int32_t num_blocks,
                                       int32_t block_size, int32_t shared, int32_t *d_free, const int64_t *d_free_at,
                                       int64_t *d_free_at_out, int32_t *d_ctx_out, int32_t *d_q_start,
                                       int32_t total_rows, int32_t *d_positions, int64_t *d_slots, int32_t *d_status,
                                       kvi_stream_t stream)
{
    if (R < 1 || R > KVI_MAX_REQUESTS) return arg_error("R=%d outside [1, %d]", R, KVI_MAX_REQUESTS);
    if (num_blocks < 1 || block_size < 1 || max_blocks < 1)
        return arg_error("num_blocks, block_size and max_blocks must be >= 1");
    if (shared < 0 || shared % block_size || shared / block_size > max_blocks)
        return arg_error("shared=%d must be whole blocks of %d, max_blocks=%d at most", shared, block_size, max_blocks);
    if (total_rows < 0) return arg_error("total_rows=%d must be >= 0", total_rows);
    if (unusable(d_ctx_lens, 4) || unusable(d_new_lens, 4) || unusable(d_block_tables, 4) || unusable(d_free, 4) ||
        unusable(d_free_at, 8) || unusable(d_free_at_out, 8) || unusable(d_ctx_out, 4) || unusable(d_q_start, 4) ||
        unusable(d_status, 4) || (total_rows && (unusable(d_positions, 4) || unusable(d_slots, 8))))
        return arg_error("a required pointer is NULL or misaligned");
    if (d_ctx_out == d_ctx_lens || d_ctx_out == d_new_lens || d_free_at_out == d_free_at)
        return arg_error("ctx_out and free_at_out must be other buffers than the inputs");
    BatchParams p{};
    p.R = R;
    p.ctx_lens = d_ctx_lens;
    p.new_lens = d_new_lens;
    p.tables = d_block_tables;
    p.max_blocks = max_blocks;
    p.num_blocks = num_blocks;
    p.B = block_size;
    p.shared = shared;
    p.free_ids = d_free;
    p.free_at = d_free_at;
    p.free_at_out = d_free_at_out;
    p.ctx_out = d_ctx_out;
    p.q_start = d_q_start;
    p.total_rows = total_rows;
    p.positions = d_positions;
    p.slots = d_slots;
    p.status = d_status;
    return cuda_status(R <= 256 ? run_batch<256>(p, stream) : run_batch<512>(p, stream), "kvi_batch_tables");
}
