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
// requests by itself (48 KB at most, from L2): no block waits for another, and a
// step is one launch without a workspace.  What bounds it is that chain of
// latencies (lengths, two scans, a search, a block's number, a store).
#include <cuda_runtime.h>

#include <algorithm>

#include "kvi_attn.cuh"

namespace kvi {

namespace {

constexpr int kBatchThreads = 256, kBatchWarps = kBatchThreads / 32;
constexpr int kRowsPerThread = 4;

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

// Exclusive sums of a over the block's threads, and the sum of all.
__device__ __forceinline__ int64_t block_scan(int64_t a, int64_t *s_warp, int64_t &all)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t sum = a;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += u;
    }
    if (lane == 31) s_warp[warp] = sum;
    __syncthreads();
    int64_t before = 0;
    all = 0;
#pragma unroll
    for (int w = 0; w < kBatchWarps; ++w) {
        if (w < warp) before += s_warp[w];
        all += s_warp[w];
    }
    __syncthreads();
    return before + sum - a;
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

// What a request asks for, by its own numbers alone.
struct Ask {
    int32_t ctx, n;     // n < 0: finished
    int32_t had, need;  // blocks it has and needs
    int32_t back;       // blocks that go back to the ring
    bool good;
};
__device__ __forceinline__ Ask ask_of(const BatchParams &p, int r, bool report)
{
    Ask a;
    a.ctx = p.ctx_lens[r];
    a.n = p.new_lens[r];
    const int64_t room = (int64_t)p.max_blocks * p.B, end = (int64_t)a.ctx + max(a.n, 0);
    int err = 0;
    if (a.ctx < 0 || a.ctx > room || (a.n > 0 && a.ctx < p.shared)) err = KVI_ERR_OUT_OF_RANGE;
    else if (end > room || end > INT32_MAX) err = KVI_ERR_CAPACITY;
    a.good = err == 0;
    if (err && report) record_status(p.status, err);
    a.had = a.good ? (int32_t)(((int64_t)a.ctx + p.B - 1) / p.B) : 0;
    a.need = a.good && a.n > 0 ? (int32_t)((end + p.B - 1) / p.B) - a.had : 0;
    a.back = a.good && a.n < 0 ? max(0, a.had - p.shared / p.B) : 0;
    return a;
}

__global__ void __launch_bounds__(kBatchThreads) batch_kernel(const __grid_constant__ BatchParams p)
{
    extern __shared__ int32_t s_all[];
    int32_t *s_start = s_all, *s_back = s_start + p.R + 1, *s_ctx = s_back + p.R + 1, *s_need = s_ctx + p.R;
    __shared__ int64_t s_warp[kBatchWarps];
    const int tid = threadIdx.x;
    const bool first = blockIdx.x == 0;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t head = p.free_at[0], tail = p.free_at[1];
    const bool ring = head >= 0 && tail >= head && tail - head <= p.num_blocks;
    const int64_t avail = ring ? tail - head : 0;
    if (!ring && first && tid == 0) record_status(p.status, KVI_ERR_OUT_OF_RANGE);

    // ---- what is asked for, in the requests' order
    const int per = (p.R + kBatchThreads - 1) / kBatchThreads, r0 = min(p.R, tid * per), r1 = min(p.R, r0 + per);
    int64_t need = 0, rows = 0, back = 0;
    for (int r = r0; r < r1; ++r) {
        const Ask a = ask_of(p, r, first);
        need += a.need;
        rows += a.good ? max(a.n, 0) : 0;
        back += a.back;
    }
    int64_t all_need, all_rows, all_back;
    int64_t need_at = block_scan(need, s_warp, all_need), rows_at = block_scan(rows, s_warp, all_rows);
    int64_t back_at = block_scan(back, s_warp, all_back);
    const bool returns = ring && all_back <= p.num_blocks - avail;
    if (!returns && ring && first && tid == 0) record_status(p.status, KVI_ERR_CAPACITY);

    // ---- what is granted: in order while blocks and rows last
    int64_t granted = 0;
    const bool plenty = all_need <= avail && all_rows <= p.total_rows;
    {
        int64_t nd = need_at, rw = rows_at;
        for (int r = r0; r < r1 && !plenty; ++r) {
            const Ask a = ask_of(p, r, false);
            const int n = a.good ? max(a.n, 0) : 0;
            nd += a.need;
            rw += n;
            if (n > 0 && (a.need == 0 || nd <= avail) && rw <= p.total_rows)
                granted += n;
            else if (n > 0 && first)
                record_status(p.status, KVI_ERR_CAPACITY);
        }
        if (plenty) granted = rows;
    }
    int64_t all_granted = all_rows, at = rows_at;
    if (!plenty) at = block_scan(granted, s_warp, all_granted);
    int64_t taken = 0;
    for (int r = r0; r < r1; ++r) {
        const Ask a = ask_of(p, r, false);
        const int n = a.good ? max(a.n, 0) : 0;
        rows_at += n;
        const bool got = n > 0 && (a.need == 0 || need_at + a.need <= avail) && rows_at <= p.total_rows;
        s_start[r] = (int32_t)at;
        s_back[r] = (int32_t)min(back_at, (int64_t)INT32_MAX);
        s_ctx[r] = a.ctx;
        s_need[r] = got ? (int32_t)need_at : 0;
        if (first) {
            p.q_start[r] = (int32_t)at;
            p.ctx_out[r] = a.n < 0 && a.good && returns ? 0 : got ? a.ctx + n : a.ctx;
        }
        if (got) {
            at += n;
            taken += a.need;
        }
        need_at += a.need;
        back_at += a.back;
    }
    if (tid == 0) {
        s_start[p.R] = (int32_t)all_granted;
        s_back[p.R] = returns ? (int32_t)all_back : 0;
        if (first) p.q_start[p.R] = (int32_t)all_granted;
    }
    int64_t all_taken = all_need;
    if (!plenty) (void)block_scan(taken, s_warp, all_taken);
    if (first && tid == 0) {
        p.free_at_out[0] = head + (ring ? all_taken : 0);
        p.free_at_out[1] = tail + (returns ? all_back : 0);
    }
    __syncthreads();

    // ---- rows: slots and positions, and the tables' new entries
    const int32_t real = s_start[p.R], head_in = ring ? (int32_t)(head % p.num_blocks) : 0;
    const int64_t stride = (int64_t)gridDim.x * kBatchThreads;
    for (int64_t row = (int64_t)blockIdx.x * kBatchThreads + tid; row < p.total_rows; row += stride) {
        int32_t pos = 0;
        int64_t slot = -1;
        if (row < real) {
            const int r = last_at_most(s_start, p.R, (int32_t)row);
            const int32_t ctx = s_ctx[r];
            pos = ctx + ((int32_t)row - s_start[r]);
            const int32_t col = pos / p.B, off = pos - col * p.B;
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
    // ---- finished requests' blocks
    const int32_t returned = s_back[p.R], tail_in = ring ? (int32_t)(tail % p.num_blocks) : 0;
    for (int64_t i = (int64_t)blockIdx.x * kBatchThreads + tid; i < returned; i += stride) {
        const int r = last_at_most(s_back, p.R, (int32_t)i);
        int64_t to = (int64_t)tail_in + i;
        if (to >= p.num_blocks) to -= p.num_blocks;
        p.free_ids[to] = p.tables[(int64_t)r * p.max_blocks + p.shared / p.B + ((int32_t)i - s_back[r])];
    }
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
    const int bytes = (4 * R + 2) * 4;
    const cudaError_t e = smem_opt_in(batch_kernel, (4 * KVI_MAX_REQUESTS + 2) * 4);
    if (e != cudaSuccess) return cuda_status(e, "kvi_batch_tables");
    const int64_t wanted = std::max<int64_t>((total_rows + (int64_t)kBatchThreads * kRowsPerThread - 1) /
                                                 (kBatchThreads * kRowsPerThread),
                                             R / 32);
    const unsigned grid = (unsigned)std::min<int64_t>(std::max<int64_t>(wanted, 1), kPlanSms);
    return cuda_status(launch_chained(batch_kernel, dim3(grid), kBatchThreads, bytes, stream, p), "kvi_batch_tables");
}
