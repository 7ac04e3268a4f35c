// kvi_cache4.cu -- the 4-bit paged cache: rows in (kvi_cache4_write), rows
// out (kvi_cache4_read) and the cut to a budget (kvi_cache4_evict).
//
// A row of one KV head is D / 32 groups of 32 channels: step = bf16(max |x| /
// 7), code = x / step rounded to the nearest integer, ties to even.  Both
// divisions are IEEE float32; step rounds once more, to bf16, because a
// step of 16 bits per 32 codes is what makes the format 4.5 bits, and the
// codes are taken against the rounded step, so that no error of it is left
// in them.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdarg>
#include <cstdio>

#include "kvi_attn.cuh"

namespace kvi {

namespace {

// ------------------------------------------------------------ rows in and out
//
// A thread owns four neighbouring channels of one token and head: the four
// nibbles of one 16-bit piece of both code layouts.  Eight neighbouring lanes
// hold a group.

struct RowParams {
    const __nv_bfloat16 *k_in, *v_in;
    __nv_bfloat16 *k_out, *v_out;
    int64_t k_stride, v_stride;  // elements between rows
    const int64_t *slots;
    int64_t T, n_slots;
    int32_t H, D;
    Page4 page;
    uint8_t *pool;
    int32_t *status;
};

constexpr int kRowThreads = 256;

// The 16-bit pieces of channels 32 g + 4 s .. + 3 of the token at `off`.
__device__ __forceinline__ int64_t k_piece(const Page4 &pg, int off, int g, int s)
{
    return (int64_t)off * (pg.D / 2) + (((s >> 1) * pg.groups() + g) * 4) + (s & 1) * 2;
}
__device__ __forceinline__ int64_t v_piece(const Page4 &pg, int off, int g, int s)
{
    return pg.v_codes() + (int64_t)(off >> 1) * pg.D + ((s * pg.groups() + g) * 4) + (off & 1) * 2;
}
__device__ __forceinline__ int64_t k_step_at(const Page4 &pg, int off, int g)
{
    return pg.k_steps() + ((int64_t)off * pg.groups() + g) * 2;
}
__device__ __forceinline__ int64_t v_step_at(const Page4 &pg, int off, int g)
{
    return pg.v_steps() + (((int64_t)(off >> 1) * pg.groups() + g) * 2 + (off & 1)) * 2;
}

// Step and four codes of this lane's channels; the eight lanes of a group
// agree on the step.
__device__ __forceinline__ void quantise4(uint2 raw, uint16_t &step, uint16_t &codes)
{
    // |x| as bf16 bits: their order is that of the values, infinities and
    // NaN at the top
    uint32_t top = max(max(raw.x & 0x7fffu, (raw.x >> 16) & 0x7fffu), max(raw.y & 0x7fffu, (raw.y >> 16) & 0x7fffu));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (top >= 0x7f80u) {  // not finite: the whole group reads back as NaN
        step = 0x7fff;
        codes = 0x8888;
        return;
    }
    const __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(__uint_as_float(top << 16), 7.0f));
    step = __bfloat16_as_ushort(sb);
    const float sf = __bfloat162float(sb);
    const float x[4] = {bf16_lo(raw.x), bf16_hi(raw.x), bf16_lo(raw.y), bf16_hi(raw.y)};
    uint32_t c = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        // sf == 0: 0 / 0 or x / 0 where x is too small for any bf16 step
        float q = sf > 0.f ? rintf(__fdiv_rn(x[j], sf)) : 0.f;
        // the step rounds down by at most 2^-9 of itself (less exactly for
        // subnormal steps), so only there a quotient can pass 7
        q = fminf(fmaxf(q, -7.f), 7.f);
        c |= (uint32_t)((int)q + 8) << (4 * j);
    }
    codes = (uint16_t)c;
}

__global__ void __launch_bounds__(kRowThreads) cache4_write_kernel(const RowParams p)
{
    const int quads = p.D / 4;
    const int64_t per_row = (int64_t)p.H * quads;  // a multiple of 8: a group never leaves its warp
    const int64_t n = p.T * per_row;
    const int64_t i = (int64_t)blockIdx.x * kRowThreads + threadIdx.x;
    const bool in = i < n;
    const int64_t t = in ? i / per_row : 0;
    const int rest = (int)(in ? i % per_row : 0);
    const int h = rest / quads, q = rest % quads;
    const int64_t slot = in ? p.slots[t] : -1;
    const bool live = slot >= 0 && slot < p.n_slots;
    if (slot >= p.n_slots && rest == 0) record_status(p.status, KVI_ERR_OUT_OF_RANGE);
    uint2 kr = make_uint2(0, 0), vr = make_uint2(0, 0);
    if (live) {
        kr = *reinterpret_cast<const uint2 *>(p.k_in + t * p.k_stride + (int64_t)h * p.D + 4 * q);
        vr = *reinterpret_cast<const uint2 *>(p.v_in + t * p.v_stride + (int64_t)h * p.D + 4 * q);
    }
    uint16_t ks, kc, vs, vc;
    quantise4(kr, ks, kc);
    quantise4(vr, vs, vc);
    if (!live) return;
    const int off = (int)(slot % p.page.B), g = q >> 3, s = q & 7;
    uint8_t *page = p.pool + ((slot / p.page.B) * p.H + h) * p.page.bytes();
    *reinterpret_cast<uint16_t *>(page + k_piece(p.page, off, g, s)) = kc;
    *reinterpret_cast<uint16_t *>(page + v_piece(p.page, off, g, s)) = vc;
    if (s == 0) {
        *reinterpret_cast<uint16_t *>(page + k_step_at(p.page, off, g)) = ks;
        *reinterpret_cast<uint16_t *>(page + v_step_at(p.page, off, g)) = vs;
    }
}

// step * code: exact in float32 (8 by 4 bits), rounded once to bf16
__device__ __forceinline__ uint2 values4(uint16_t step, uint32_t codes)
{
    const float s = __uint_as_float((uint32_t)step << 16);
    float x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = s * (float)((int)((codes >> (4 * j)) & 15u) - 8);
    return make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
}

__global__ void __launch_bounds__(kRowThreads) cache4_read_kernel(const RowParams p)
{
    const int quads = p.D / 4;
    const int64_t per_row = (int64_t)p.H * quads;
    const int64_t i = (int64_t)blockIdx.x * kRowThreads + threadIdx.x;
    if (i >= p.T * per_row) return;
    const int64_t t = i / per_row;
    const int rest = (int)(i % per_row);
    const int h = rest / quads, q = rest % quads;
    const int64_t slot = p.slots[t];
    if (slot >= p.n_slots && rest == 0) record_status(p.status, KVI_ERR_OUT_OF_RANGE);
    if (slot < 0 || slot >= p.n_slots) return;
    const int off = (int)(slot % p.page.B), g = q >> 3, s = q & 7;
    const uint8_t *page = p.pool + ((slot / p.page.B) * p.H + h) * p.page.bytes();
    const uint2 k = values4(*reinterpret_cast<const uint16_t *>(page + k_step_at(p.page, off, g)),
                            *reinterpret_cast<const uint16_t *>(page + k_piece(p.page, off, g, s)));
    const uint2 v = values4(*reinterpret_cast<const uint16_t *>(page + v_step_at(p.page, off, g)),
                            *reinterpret_cast<const uint16_t *>(page + v_piece(p.page, off, g, s)));
    *reinterpret_cast<uint2 *>(p.k_out + t * p.k_stride + (int64_t)h * p.D + 4 * q) = k;
    *reinterpret_cast<uint2 *>(p.v_out + t * p.v_stride + (int64_t)h * p.D + 4 * q) = v;
}

// ----------------------------------------------------------------- eviction
//
// Per request and head: the budget-th largest rank is found 11 bits at a time
// (three counting passes over the ranks), then one ordered pass marks the kept
// slots (ties in slot order) and lists the freed slots below the budget and
// the kept ones above it.  Both lists have the same length; the second
// kernel copies row for row.

struct EvictParams {
    int32_t R, H, budget, sink, recent;
    const int32_t *ctx_lens;
    int32_t max_ctx, max_blocks;
    const int32_t *block_tables;
    int32_t num_blocks;
    Page4 page;
    uint8_t *pool;
    const float *w;
    const int32_t *pos;
    int64_t stride;
    float *w_out;
    int32_t *pos_out;
    int32_t *ctx_out;
    int32_t *holes, *tails;  // [R][H][most] slots
    int32_t *moves;          // [R][H]
    int32_t most;            // moves a row can need
    int32_t cap;             // ranks kept in shared memory
    int32_t *status;
};

constexpr int kEvictThreads = 1024;
constexpr int kMoveThreads = 256;
constexpr int kBins = 2048;           // two per thread
constexpr int kRankCap = 24 * 1024;   // ranks kept in shared memory (two blocks fit an SM)

// Rank order of a slot as an unsigned number: protected slots first, then
// by weight (-0 as 0, NaN above infinity).
__device__ __forceinline__ uint32_t evict_rank(float w, int pos, int sink, int64_t newest_from)
{
    if (pos < sink || (int64_t)pos >= newest_from) return 0xffffffffu;
    if (w != w) return 0xfffffffeu;
    const uint32_t b = __float_as_uint(w + 0.0f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Sum of v over the threads before this one.
__device__ __forceinline__ int block_sum_before(int v, int *warp_sums)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int sum = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += u;
    }
    if (lane == 31) warp_sums[warp] = sum;
    __syncthreads();
    int before = lane < warp ? warp_sums[lane] : 0;
    before = __reduce_add_sync(0xffffffffu, before);
    return before + sum - v;
}

// Exclusive prefix sum over the block of a 0/1 flag; `total` for everybody.
__device__ __forceinline__ int block_rank(bool flag, int *warp_sums, int &total)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t votes = __ballot_sync(0xffffffffu, flag);
    __syncthreads();  // the last call's sums have been read
    if (lane == 0) warp_sums[warp] = __popc(votes);
    __syncthreads();
    if (warp == 0) {
        const int v = warp_sums[lane];
        int sum = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += u;
        }
        warp_sums[lane] = sum - v;
        if (lane == 31) warp_sums[32] = sum;
    }
    __syncthreads();
    total = warp_sums[32];
    return warp_sums[warp] + __popc(votes & ((1u << lane) - 1u));
}

__global__ void __launch_bounds__(kEvictThreads) evict_select_kernel(const EvictParams p)
{
    extern __shared__ uint32_t s_rank[];  // of the first p.cap slots
    __shared__ int s_warp[33];
    __shared__ int s_hist[kBins];
    __shared__ int s_newest, s_digit, s_left;
    const int h = blockIdx.x % p.H, r = blockIdx.x / p.H, tid = threadIdx.x;
    const int64_t row = (int64_t)blockIdx.x;
    const float *w = p.w + row * p.stride;
    const int32_t *pos = p.pos + row * p.stride;
    float *w_out = p.w_out + row * p.stride;
    int32_t *pos_out = p.pos_out + row * p.stride;
    const int n = p.ctx_lens[r];
    pdl_launch_dependents();
    if (n < 0 || n > p.max_ctx || (int64_t)n > (int64_t)p.max_blocks * p.page.B) {
        if (tid == 0) {
            record_status(p.status, KVI_ERR_OUT_OF_RANGE);
            p.moves[row] = 0;
        }
        return;
    }
    const int left = min(n, p.budget);
    if (h == 0 && tid == 0) p.ctx_out[r] = left;
    if (n <= p.budget) {
        for (int i = tid; i < n; i += kEvictThreads) {
            w_out[i] = w[i];
            pos_out[i] = pos[i];
        }
        if (tid == 0) p.moves[row] = 0;
        return;
    }
    if (tid == 0) s_newest = INT32_MIN;
    for (int i = tid; i < kBins; i += kEvictThreads) s_hist[i] = 0;
    __syncthreads();
    int newest = INT32_MIN;
    for (int i = tid; i < n; i += kEvictThreads) newest = max(newest, pos[i]);
    newest = __reduce_max_sync(0xffffffffu, newest);
    if ((tid & 31) == 0) atomicMax(&s_newest, newest);
    __syncthreads();
    const int64_t from = (int64_t)s_newest - p.recent + 1;
    auto rank_of = [&](int i) { return i < p.cap ? s_rank[i] : evict_rank(w[i], pos[i], p.sink, from); };

    // the budget-th largest rank, 11, 11 and 10 bits at a time from the top
    uint32_t found = 0;
    int want = p.budget;  // of the slots that share the bits found so far
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t mask = pass == 2 ? 1023u : 2047u;
        for (int i = tid; i < n; i += kEvictThreads) {
            uint32_t k;
            if (pass == 0) {
                k = evict_rank(w[i], pos[i], p.sink, from);
                if (i < p.cap) s_rank[i] = k;
            } else {
                k = rank_of(i);
                if ((k ^ found) >> (pass == 1 ? 21 : 10)) continue;
            }
            atomicAdd(&s_hist[(k >> shift) & mask], 1);
        }
        __syncthreads();
        // from the top bin down, two bins a thread: the one where the count
        // passes `want`
        const int hi = kBins - 1 - 2 * tid;
        const int a = s_hist[hi], b = s_hist[hi - 1];
        s_hist[hi] = s_hist[hi - 1] = 0;
        const int above = block_sum_before(a + b, s_warp);
        if (above < want && above + a + b >= want) {
            s_digit = above + a >= want ? hi : hi - 1;
            s_left = want - above - (above + a >= want ? 0 : a);
        }
        __syncthreads();
        found |= (uint32_t)s_digit << shift;
        want = s_left;
    }
    // ranks above `found` stay, and the first `want` slots that equal it
    int ties = 0, n_holes = 0, n_tails = 0;
    int32_t *holes = p.holes + row * p.most, *tails = p.tails + row * p.most;
    for (int i0 = 0; i0 < n; i0 += kEvictThreads) {
        const int i = i0 + tid;
        const bool in = i < n;
        const uint32_t k = in ? rank_of(i) : 0u;
        const bool tie = in && k == found;
        int c;
        const int rank = ties + block_rank(tie, s_warp, c);
        ties += c;
        const bool keep = in && (k > found || (tie && rank < want));
        const bool hole = in && i < left && !keep, tail = keep && i >= left;
        // a block's slots lie below the budget, above it, or (once) across it
        if (i0 < left) {
            const int at = n_holes + block_rank(hole, s_warp, c);
            n_holes += c;
            if (hole) holes[at] = i;
        }
        if (i0 + kEvictThreads > left) {
            const int at = n_tails + block_rank(tail, s_warp, c);
            n_tails += c;
            if (tail) tails[at] = i;
        }
        if (in && !hole) {
            w_out[i] = i < left ? w[i] : 0.f;
            pos_out[i] = i < left ? pos[i] : -1;
        }
    }
    __syncthreads();
    for (int i = tid; i < n_holes; i += kEvictThreads) {
        w_out[holes[i]] = w[tails[i]];
        pos_out[holes[i]] = pos[tails[i]];
    }
    if (tid == 0) p.moves[row] = n_holes;
}

// One warp per moved row: 16-bit pieces, as two tokens share each word of
// the V codes and steps.
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams p)
{
    pdl_wait();
    const int64_t row = blockIdx.y;
    const int h = (int)(row % p.H), r = (int)(row / p.H), lane = threadIdx.x & 31;
    const int n = p.moves[row];
    const int32_t *table = p.block_tables + (int64_t)r * p.max_blocks;
    const int G = p.page.groups(), quads = p.page.D / 4;
    const int warps = gridDim.x * (kMoveThreads / 32);
    for (int i = blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5); i < n; i += warps) {
        const int dst = p.holes[row * p.most + i], src = p.tails[row * p.most + i];
        const int db = table[dst / p.page.B], sb = table[src / p.page.B];
        if (db < 0 || db >= p.num_blocks || sb < 0 || sb >= p.num_blocks) {
            if (lane == 0) record_status(p.status, KVI_ERR_OUT_OF_RANGE);
            continue;
        }
        uint8_t *to = p.pool + ((int64_t)db * p.H + h) * p.page.bytes();
        const uint8_t *fr = p.pool + ((int64_t)sb * p.H + h) * p.page.bytes();
        const int d = dst % p.page.B, s = src % p.page.B;
        for (int q = lane; q < quads; q += 32) {
            *reinterpret_cast<uint16_t *>(to + k_piece(p.page, d, q >> 3, q & 7)) =
                *reinterpret_cast<const uint16_t *>(fr + k_piece(p.page, s, q >> 3, q & 7));
            *reinterpret_cast<uint16_t *>(to + v_piece(p.page, d, q >> 3, q & 7)) =
                *reinterpret_cast<const uint16_t *>(fr + v_piece(p.page, s, q >> 3, q & 7));
        }
        if (lane < G) {
            *reinterpret_cast<uint16_t *>(to + k_step_at(p.page, d, lane)) =
                *reinterpret_cast<const uint16_t *>(fr + k_step_at(p.page, s, lane));
            *reinterpret_cast<uint16_t *>(to + v_step_at(p.page, d, lane)) =
                *reinterpret_cast<const uint16_t *>(fr + v_step_at(p.page, s, lane));
        }
    }
}

bool aligned16(const void *p, int64_t stride) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride % 8 == 0; }

bool page_ok(int32_t H, int32_t D, int32_t num_blocks, int32_t B)
{
    return H >= 1 && H <= 4096 && D >= 32 && D <= KVI_MAX_ATTN_HEAD_DIM && D % 32 == 0 && num_blocks >= 1 && B >= 16 &&
           B % 16 == 0 && B <= (1 << 20);
}

kvi_status check_cache4(int32_t H, int32_t D, const kvi_paged_cache *c, int32_t layer)
{
    if (!c || !c->layer_base) return arg_error("cache or cache->layer_base is NULL");
    if (!page_ok(H, D, c->num_blocks, c->block_size))
        return arg_error("4-bit cache: kv_heads=%d (1..4096), head_dim=%d (a multiple of 32 up to %d), num_blocks=%d "
                         "(>= 1), block_size=%d (a multiple of 16)",
                         H, D, KVI_MAX_ATTN_HEAD_DIM, c->num_blocks, c->block_size);
    if (layer < 0 || layer >= c->layers) return arg_error("layer=%d outside [0, %d)", layer, c->layers);
    if (!c->layer_base[layer] || reinterpret_cast<uintptr_t>(c->layer_base[layer]) % 16)
        return arg_error("layer_base[%d] is NULL or not 16-byte aligned", layer);
    return KVI_OK;
}

kvi_status rows_params(RowParams &p, int32_t H, int32_t D, const kvi_paged_cache *cache, int32_t layer, int64_t T,
                       const void *k, int64_t ks, const void *v, int64_t vs, const int64_t *slots, int32_t *status)
{
    const kvi_status st = check_cache4(H, D, cache, layer);
    if (st != KVI_OK) return st;
    if (T < 0 || unusable(status, 4)) return arg_error("T < 0, or d_status is NULL or misaligned");
    if (T && (!k || !v || unusable(slots, 8))) return arg_error("d_k, d_v and d_slots are required");
    if (T && (!aligned16(k, ks) || !aligned16(v, vs) || ks < (int64_t)H * D || vs < (int64_t)H * D))
        return arg_error("rows must be 16-byte aligned, with strides of at least kv_heads * head_dim elements");
    if (T * H * (D / 4) / kRowThreads >= 0x7fffffff) return arg_error("T=%lld rows are too many", (long long)T);
    p.k_stride = ks;
    p.v_stride = vs;
    p.slots = slots;
    p.T = T;
    p.n_slots = (int64_t)cache->num_blocks * cache->block_size;
    p.H = H;
    p.D = D;
    p.page = Page4{cache->block_size, D};
    p.pool = static_cast<uint8_t *>(cache->layer_base[layer]);
    p.status = status;
    return KVI_OK;
}

unsigned row_blocks(const RowParams &p)
{
    return (unsigned)((p.T * p.H * (p.D / 4) + kRowThreads - 1) / kRowThreads);
}

size_t evict_bytes(int32_t H, int32_t R, int32_t max_ctx, int32_t *most)
{
    // a row moves at most min(budget, ctx - budget) <= ctx / 2 keys
    *most = std::max(1, max_ctx / 2);
    return (((size_t)R * H * (*most) * 4 + 255) & ~(size_t)255) * 2 + (((size_t)R * H * 4 + 255) & ~(size_t)255);
}

}  // namespace

kvi_status cache4_check(int32_t H, int32_t D, const kvi_paged_cache *c, int32_t layer)
{
    return check_cache4(H, D, c, layer);
}

}  // namespace kvi

using namespace kvi;

extern "C" size_t kvi_cache4_layer_bytes(int32_t kv_heads, int32_t head_dim, int32_t num_blocks, int32_t block_size)
{
    if (!page_ok(kv_heads, head_dim, num_blocks, block_size)) return 0;
    return (size_t)num_blocks * kv_heads * (size_t)Page4{block_size, head_dim}.bytes();
}

extern "C" kvi_status kvi_cache4_write(int32_t kv_heads, int32_t head_dim, const kvi_paged_cache *cache, int32_t layer,
                                       int64_t T, const void *d_k, int64_t k_row_stride, const void *d_v,
                                       int64_t v_row_stride, const int64_t *d_slots, int32_t *d_status,
                                       kvi_stream_t stream)
{
    RowParams p{};
    const kvi_status st = rows_params(p, kv_heads, head_dim, cache, layer, T, d_k, k_row_stride, d_v, v_row_stride,
                                      d_slots, d_status);
    if (st != KVI_OK || T == 0) return st;
    p.k_in = static_cast<const __nv_bfloat16 *>(d_k);
    p.v_in = static_cast<const __nv_bfloat16 *>(d_v);
    cache4_write_kernel<<<row_blocks(p), kRowThreads, 0, stream>>>(p);
    return cuda_status(cudaGetLastError(), "kvi_cache4_write");
}

extern "C" kvi_status kvi_cache4_read(int32_t kv_heads, int32_t head_dim, const kvi_paged_cache *cache, int32_t layer,
                                      int64_t T, const int64_t *d_slots, void *d_k, int64_t k_row_stride, void *d_v,
                                      int64_t v_row_stride, int32_t *d_status, kvi_stream_t stream)
{
    RowParams p{};
    const kvi_status st = rows_params(p, kv_heads, head_dim, cache, layer, T, d_k, k_row_stride, d_v, v_row_stride,
                                      d_slots, d_status);
    if (st != KVI_OK || T == 0) return st;
    p.k_out = static_cast<__nv_bfloat16 *>(d_k);
    p.v_out = static_cast<__nv_bfloat16 *>(d_v);
    cache4_read_kernel<<<row_blocks(p), kRowThreads, 0, stream>>>(p);
    return cuda_status(cudaGetLastError(), "kvi_cache4_read");
}

extern "C" size_t kvi_cache4_evict_workspace_bytes(int32_t kv_heads, int32_t R, int32_t max_ctx)
{
    int32_t most;
    if (kv_heads < 1 || kv_heads > 4096 || R < 1 || R > KVI_MAX_REQUESTS || max_ctx < 0) return 0;
    return evict_bytes(kv_heads, R, max_ctx, &most);
}

extern "C" kvi_status kvi_cache4_evict(int32_t kv_heads, int32_t head_dim, int32_t R, const kvi_paged_cache *cache,
                                       int32_t layer, const int32_t *d_ctx_lens, int32_t max_ctx,
                                       const int32_t *d_block_tables, int32_t max_blocks, int32_t budget, int32_t sink,
                                       int32_t recent, const float *d_weights, const int32_t *d_pos, int64_t stride,
                                       float *d_weights_out, int32_t *d_pos_out, int32_t *d_ctx_out, void *d_ws,
                                       size_t ws_bytes, int32_t *d_status, kvi_stream_t stream)
{
    kvi_status st = check_cache4(kv_heads, head_dim, cache, layer);
    if (st != KVI_OK) return st;
    st = check_pages(cache, layer, R, max_blocks, d_block_tables);
    if (st != KVI_OK) return st;
    if ((int64_t)R * kv_heads > 65535) return arg_error("R * kv_heads = %lld is above 65535", (long long)R * kv_heads);
    for (const void *q : {(const void *)d_ctx_lens, (const void *)d_weights, (const void *)d_pos,
                          (const void *)d_weights_out, (const void *)d_pos_out, (const void *)d_ctx_out,
                          (const void *)d_ws, (const void *)d_status})
        if (unusable(q, 4)) return arg_error("a required pointer is NULL or misaligned");
    if (d_weights == d_weights_out || d_pos == d_pos_out || d_ctx_lens == d_ctx_out)
        return arg_error("the outputs must be other buffers than the inputs");
    if (max_ctx < 0 || stride < max_ctx) return arg_error("max_ctx=%d, stride=%lld", max_ctx, (long long)stride);
    if (budget < 1 || sink < 0 || recent < 0 || (int64_t)sink + recent > budget)
        return arg_error("budget=%d (>= 1), sink=%d and recent=%d (>= 0, together at most the budget)", budget, sink,
                         recent);
    EvictParams p{};
    const size_t need = evict_bytes(kv_heads, R, max_ctx, &p.most);
    if (ws_bytes < need || reinterpret_cast<uintptr_t>(d_ws) % 256)
        return arg_error("workspace of %zu bytes (256-byte aligned) needed, %zu given", need, ws_bytes);
    p.R = R;
    p.H = kv_heads;
    p.budget = budget;
    p.sink = sink;
    p.recent = recent;
    p.ctx_lens = d_ctx_lens;
    p.max_ctx = max_ctx;
    p.max_blocks = max_blocks;
    p.block_tables = d_block_tables;
    p.num_blocks = cache->num_blocks;
    p.page = Page4{cache->block_size, head_dim};
    p.pool = static_cast<uint8_t *>(cache->layer_base[layer]);
    p.w = d_weights;
    p.pos = d_pos;
    p.stride = stride;
    p.w_out = d_weights_out;
    p.pos_out = d_pos_out;
    p.ctx_out = d_ctx_out;
    const size_t list = ((size_t)R * kv_heads * p.most * 4 + 255) & ~(size_t)255;
    p.holes = static_cast<int32_t *>(d_ws);
    p.tails = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(d_ws) + list);
    p.moves = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(d_ws) + 2 * list);
    p.status = d_status;
    p.cap = std::min(max_ctx, kRankCap);
    cudaError_t e = smem_opt_in(evict_select_kernel, kRankCap * 4);
    if (e != cudaSuccess) return cuda_status(e, "kvi_cache4_evict");
    evict_select_kernel<<<(unsigned)(R * kv_heads), kEvictThreads, (size_t)p.cap * 4, stream>>>(p);
    st = cuda_status(cudaGetLastError(), "kvi_cache4_evict");
    if (st != KVI_OK || max_ctx <= budget) return st;  // nothing can move
    // enough warps that none copies more than a few rows, without a grid of
    // mostly idle blocks where many heads share the GPU
    const int rows = std::min(p.most, budget);
    const int want = std::max(1, 4096 / (R * kv_heads));
    const unsigned gx = (unsigned)std::min((rows + kMoveThreads / 32 - 1) / (kMoveThreads / 32), want);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(gx, (unsigned)(R * kv_heads));
    cfg.blockDim = dim3(kMoveThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, evict_move_kernel, p);
    return cuda_status(e != cudaSuccess ? e : cudaGetLastError(), "kvi_cache4_evict");
}
