// kvi_cache4.cu -- the 4-bit paged cache: rows in (kvi_cache4_write), rows
// out (kvi_cache4_read) and the cut to a budget (kvi_cache4_evict).
//
// A row of one KV head is D / 32 groups of 32 channels: step = bf16(max |x| /
// 7), code = x / step rounded to the nearest integer, ties to even.  The
// first division is IEEE float32 and rounds once more, to bf16, because a
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
// A thread owns eight neighbouring channels of one head of two rows, four
// neighbouring lanes a group.  Two rows, because tokens 2 i and 2 i + 1 share
// the words of V: where the two rows go to such a pair of slots, which is the
// rule for rows of a prefix, every store is a whole word; any other two rows are
// written piece by piece.
//
// Codes without a division.  x / step is wanted rounded to the nearest integer,
// ties to even, and x and step have 8 significant bits each.  So |x / step| >=
// 1/2 is either a half-integer exactly or at least 2^-10 from one: with x =
// X 2^a, step = S 2^b (128 <= S < 256) and 2 X 2^a - h S 2^b != 0 for an odd h,
// that difference is at least 2^(b - 1), and divided by 2 S 2^b at least 2^-10.
// x * (1 / step) in float32 is off by less than 2^-19 here; rounded to
// multiples of 2^-12 (by adding 3072) it is the half-integer again where the
// quotient is one, and on the same side as the quotient everywhere else.  The
// integer then falls out of a second addition, of a number with a last place
// of 1.  Likewise max / 7 is max * (1 / 7) rounded to bf16: 7 times the middle of
// two neighbouring bf16 numbers is at least 2^-12 of itself from any bf16 number.
// Steps too small for their reciprocal take a division.

struct RowParams {
    const __nv_bfloat16 *k_in, *v_in;
    __nv_bfloat16 *k_out, *v_out;
    int64_t k_stride, v_stride;  // elements between rows
    const int64_t *slots;
    int64_t T, n_slots;
    int32_t H, D;
    int32_t heads_apart;         // a thread takes the heads h, h + heads_apart, ..
    int32_t lanes;               // heads_apart * D / 8: threads of a pair of rows
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

// Step and eight codes (channel n in nibble n) of this lane's channels; the
// four lanes of a group (`group`, of the warp's) agree on the step.
__device__ __forceinline__ uint32_t quantise8(const uint4 &raw, uint32_t group, uint32_t &step)
{
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    // the largest |x| of both halves of the words; infinities and NaN win
    __nv_bfloat162 m = __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&w[0]));
#pragma unroll
    for (int j = 1; j < 4; ++j) m = __hmax2_nan(m, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&w[j])));
    const uint32_t both = *reinterpret_cast<const uint32_t *>(&m);
    uint32_t top = max(both & 0x7fffu, (both >> 16) & 0x7fffu);
    top = max(top, __shfl_xor_sync(group, top, 1));
    top = max(top, __shfl_xor_sync(group, top, 2));
    if (top >= 0x7f80u) {  // not finite: the whole group reads back as NaN
        step = 0x7fff;
        return 0x88888888u;
    }
    const __nv_bfloat16 sb = __float2bfloat16_rn(__fmul_rn(__uint_as_float(top << 16), 1.0f / 7.0f));
    step = __bfloat16_as_ushort(sb);
    const float sf = __bfloat162float(sb);
    uint32_t c = 0;
    if (sf >= 1.1754944e-38f) {  // 1 / step is finite; |x / step| < 7.03
        float inv;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(sf));
        // the bits of 12582920 + q, 0x4b400000 + 8 + q: summed up with weights
        // 16^n, and what is not codes taken off at the end
#pragma unroll
        for (int n = 7; n >= 0; --n) {
            const float x = n & 1 ? bf16_hi(w[n >> 1]) : bf16_lo(w[n >> 1]);
            const float q = __fadd_rn(__fmaf_rn(x, inv, 3072.f), 12582920.f - 3072.f);
            c = c * 16u + __float_as_uint(q);
        }
        c -= 0x4b400000u * 0x11111111u;
    } else {
#pragma unroll 1
        for (int n = 7; n >= 0; --n) {
            const float x = __uint_as_float((w[n >> 1] >> (16 * (n & 1))) << 16);
            // a subnormal step can be well below max / 7
            const float q = sf > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(x, sf)), -7.f), 7.f) : 0.f;
            c = (c << 4) | (uint32_t)((int)q + 8);
        }
    }
    return c;
}

// step * code: eight channels from the codes in nibbles 0..7, as the four
// words of a row.  The product has one rounding, to bf16.
__device__ __forceinline__ uint4 values8(uint32_t codes, uint32_t step)
{
    const uint32_t s2 = step | (step << 16);
    uint32_t v[4];  // (j, j + 4)
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = mul_bf16x2(codes_bf16x2(codes >> (4 * j)), s2);
    return make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410), __byte_perm(v[0], v[1], 0x7632),
                      __byte_perm(v[2], v[3], 0x7632));
}

// This thread's pair of rows and channels: rows 2 i - odd and + 1, where odd is
// the first slot's parity, so that runs of consecutive slots pair up.
struct RowWork {
    int64_t row;       // the first row (it or the second may lie outside [0, T))
    int32_t h, g, t;   // first head, group, 8-channel part of the group
    int64_t slot[2];   // -1: nothing to do
    int64_t page[2];
    int32_t off[2];
    bool pair;         // slots 2 n and 2 n + 1 of one page
};

// (threadIdx.x: the lane of the pair, threadIdx.y: the pair of the block)
__device__ __forceinline__ bool row_work(const RowParams &p, RowWork &o)
{
    const uint32_t lane = blockIdx.y * blockDim.x + threadIdx.x;
    const int64_t i = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool in = lane < (uint32_t)p.lanes;
    const uint32_t parts = (uint32_t)p.D / 8;
    o.h = (int32_t)(lane / parts);
    const uint32_t part = lane - (uint32_t)o.h * parts;
    o.g = (int32_t)(part >> 2);
    o.t = (int32_t)(part & 3);
    o.row = 2 * i - (p.slots[0] & 1);
    o.slot[0] = o.slot[1] = -1;
    if (in) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int64_t r = o.row + e;
            if (r < 0 || r >= p.T) continue;
            const int64_t s = p.slots[r];
            if (s >= p.n_slots) {
                if (lane == 0) record_status(p.status, KVI_ERR_OUT_OF_RANGE);
            } else if (s >= 0) {
                o.slot[e] = s;
            }
        }
    }
    o.pair = o.slot[0] >= 0 && !(o.slot[0] & 1) && o.slot[1] == o.slot[0] + 1;  // (B is even: one page)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        if (e == 1 && o.pair) {
            o.page[1] = o.page[0];
            o.off[1] = o.off[0] + 1;
            continue;
        }
        const int64_t s = max((int64_t)0, o.slot[e]);
        if (p.n_slots <= 0x7fffffff) {
            const uint32_t page = (uint32_t)s / (uint32_t)p.page.B;
            o.page[e] = page;
            o.off[e] = (int32_t)((uint32_t)s - page * (uint32_t)p.page.B);
        } else {
            o.page[e] = s / p.page.B;
            o.off[e] = (int32_t)(s % p.page.B);
        }
    }
    return o.slot[0] >= 0 || o.slot[1] >= 0;
}

// A row's pieces inside a page: byte offsets of this thread's codes and steps.
struct Pieces {
    int32_t k, ks, v, vs;
};
__device__ __forceinline__ Pieces pieces_of(const Page4 &pg, int off, int g, int t)
{
    return Pieces{(int32_t)k_piece(pg, off, g, 2 * t), (int32_t)k_step_at(pg, off, g), (int32_t)v_piece(pg, off, g, 2 * t),
                  (int32_t)v_step_at(pg, off, g)};
}

// Pairs of slots, the rule for a prefix, have a loop of their own, with one page
// pointer and no pieces (65 k rows of 8 heads of 128 channels stored and read back:
// 117 us, 5.2 TB/s, against 149 with one loop for both).  HBM bounds it, and how
// much of it is asked for at a time: with reading held to 40 registers, six blocks
// an SM, it takes those 117 us, 123 with four.
__global__ void __launch_bounds__(kRowThreads) cache4_write_kernel(const __grid_constant__ RowParams p)
{
    pdl_wait();
    pdl_launch_dependents();
    RowWork o;
    if (!row_work(p, o)) return;
    const uint32_t group = 0xfu << ((threadIdx.y * blockDim.x + threadIdx.x) & 28u);  // (lanes of one row work alike)
    const int64_t bytes = p.page.bytes();
    const int32_t col = 32 * o.g + 8 * o.t;
    const int v_next = 4 * p.page.groups();  // from a piece of V to the next four channels'
    if (o.pair) {
        const Pieces at = pieces_of(p.page, o.off[0], o.g, o.t);
        uint8_t *page = p.pool + (o.page[0] * p.H + o.h) * bytes;
        const __nv_bfloat16 *k_src = p.k_in + o.row * p.k_stride + o.h * p.D + col;
        const __nv_bfloat16 *v_src = p.v_in + o.row * p.v_stride + o.h * p.D + col;
#pragma unroll 1
        for (int h = o.h; h < p.H; h += p.heads_apart) {
            const uint4 k0 = *reinterpret_cast<const uint4 *>(k_src);
            const uint4 k1 = *reinterpret_cast<const uint4 *>(k_src + p.k_stride);
            const uint4 v0 = *reinterpret_cast<const uint4 *>(v_src);
            const uint4 v1 = *reinterpret_cast<const uint4 *>(v_src + p.v_stride);
            uint32_t s0, s1;
            uint32_t c0 = quantise8(k0, group, s0), c1 = quantise8(k1, group, s1);
            *reinterpret_cast<uint32_t *>(page + at.k) = c0;
            *reinterpret_cast<uint32_t *>(page + at.k + p.page.D / 2) = c1;
            if (o.t == 0) {
                *reinterpret_cast<uint16_t *>(page + at.ks) = (uint16_t)s0;
                *reinterpret_cast<uint16_t *>(page + at.ks + 2 * p.page.groups()) = (uint16_t)s1;
            }
            c0 = quantise8(v0, group, s0);
            c1 = quantise8(v1, group, s1);
            *reinterpret_cast<uint32_t *>(page + at.v) = __byte_perm(c0, c1, 0x5410);
            *reinterpret_cast<uint32_t *>(page + at.v + v_next) = __byte_perm(c0, c1, 0x7632);
            if (o.t == 0) *reinterpret_cast<uint32_t *>(page + at.vs) = s0 | (s1 << 16);
            k_src += p.heads_apart * p.D;
            v_src += p.heads_apart * p.D;
            page += p.heads_apart * bytes;
        }
        return;
    }
    // two rows of their own
    const Pieces at[2] = {pieces_of(p.page, o.off[0], o.g, o.t), pieces_of(p.page, o.off[1], o.g, o.t)};
    const __nv_bfloat16 *k_src = p.k_in + o.row * p.k_stride + col, *v_src = p.v_in + o.row * p.v_stride + col;
#pragma unroll 1
    for (int h = o.h; h < p.H; h += p.heads_apart) {
        uint4 k[2], v[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (o.slot[e] < 0) continue;
            k[e] = *reinterpret_cast<const uint4 *>(k_src + e * p.k_stride + h * p.D);
            v[e] = *reinterpret_cast<const uint4 *>(v_src + e * p.v_stride + h * p.D);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (o.slot[e] < 0) continue;
            uint32_t ks, vs;
            const uint32_t kc = quantise8(k[e], group, ks), vc = quantise8(v[e], group, vs);
            uint8_t *page = p.pool + (o.page[e] * p.H + h) * bytes;
            *reinterpret_cast<uint32_t *>(page + at[e].k) = kc;
            *reinterpret_cast<uint16_t *>(page + at[e].v) = (uint16_t)vc;
            *reinterpret_cast<uint16_t *>(page + at[e].v + v_next) = (uint16_t)(vc >> 16);
            if (o.t == 0) {
                *reinterpret_cast<uint16_t *>(page + at[e].ks) = (uint16_t)ks;
                *reinterpret_cast<uint16_t *>(page + at[e].vs) = (uint16_t)vs;
            }
        }
    }
}

__global__ void __launch_bounds__(kRowThreads, 6) cache4_read_kernel(const __grid_constant__ RowParams p)
{
    pdl_wait();
    pdl_launch_dependents();
    RowWork o;
    if (!row_work(p, o)) return;
    const int64_t bytes = p.page.bytes();
    const int32_t col = 32 * o.g + 8 * o.t;
    const int v_next = 4 * p.page.groups();
    if (o.pair) {
        const Pieces at = pieces_of(p.page, o.off[0], o.g, o.t);
        const uint8_t *page = p.pool + (o.page[0] * p.H + o.h) * bytes;
        __nv_bfloat16 *k_dst = p.k_out + o.row * p.k_stride + o.h * p.D + col;
        __nv_bfloat16 *v_dst = p.v_out + o.row * p.v_stride + o.h * p.D + col;
#pragma unroll 1
        for (int h = o.h; h < p.H; h += p.heads_apart) {
            const uint32_t k0 = *reinterpret_cast<const uint32_t *>(page + at.k);
            const uint32_t k1 = *reinterpret_cast<const uint32_t *>(page + at.k + p.page.D / 2);
            const uint32_t a = *reinterpret_cast<const uint32_t *>(page + at.v);
            const uint32_t b = *reinterpret_cast<const uint32_t *>(page + at.v + v_next);
            const uint32_t s0 = *reinterpret_cast<const uint16_t *>(page + at.ks);
            const uint32_t s1 = *reinterpret_cast<const uint16_t *>(page + at.ks + 2 * p.page.groups());
            const uint32_t s = *reinterpret_cast<const uint32_t *>(page + at.vs);
            *reinterpret_cast<uint4 *>(k_dst) = values8(k0, s0);
            *reinterpret_cast<uint4 *>(k_dst + p.k_stride) = values8(k1, s1);
            *reinterpret_cast<uint4 *>(v_dst) = values8(__byte_perm(a, b, 0x5410), s & 0xffffu);
            *reinterpret_cast<uint4 *>(v_dst + p.v_stride) = values8(__byte_perm(a, b, 0x7632), s >> 16);
            k_dst += p.heads_apart * p.D;
            v_dst += p.heads_apart * p.D;
            page += p.heads_apart * bytes;
        }
        return;
    }
    const Pieces at[2] = {pieces_of(p.page, o.off[0], o.g, o.t), pieces_of(p.page, o.off[1], o.g, o.t)};
    __nv_bfloat16 *k_dst = p.k_out + o.row * p.k_stride + col, *v_dst = p.v_out + o.row * p.v_stride + col;
#pragma unroll 1
    for (int h = o.h; h < p.H; h += p.heads_apart) {
        uint32_t kc[2], ks[2], vc[2], vs[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (o.slot[e] < 0) continue;
            const uint8_t *page = p.pool + (o.page[e] * p.H + h) * bytes;
            kc[e] = *reinterpret_cast<const uint32_t *>(page + at[e].k);
            vc[e] = *reinterpret_cast<const uint16_t *>(page + at[e].v) |
                    (uint32_t)*reinterpret_cast<const uint16_t *>(page + at[e].v + v_next) << 16;
            ks[e] = *reinterpret_cast<const uint16_t *>(page + at[e].ks);
            vs[e] = *reinterpret_cast<const uint16_t *>(page + at[e].vs);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (o.slot[e] < 0) continue;
            *reinterpret_cast<uint4 *>(k_dst + e * p.k_stride + h * p.D) = values8(kc[e], ks[e]);
            *reinterpret_cast<uint4 *>(v_dst + e * p.v_stride + h * p.D) = values8(vc[e], vs[e]);
        }
    }
}

// ----------------------------------------------------------------- eviction
//
// Per request and head: the budget-th largest rank is found 11 bits at a time
// (three counting passes over the ranks), then one ordered pass marks the kept
// slots (ties in slot order) and lists the freed slots below the budget and
// the kept ones above it.  Both lists have the same length; the rows are moved
// by the same block, or, where heads are few and rows many, by a second kernel.

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
    int32_t move_here;       // the rows are moved by the block that found them
    int32_t *status;
};

constexpr int kMoveThreads = 256;
constexpr int kBins = 2048;
constexpr int kRankCap = 24 * 1024;   // ranks kept in shared memory

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
    int before = lane < warp ? warp_sums[lane] : 0;  // warp < 32
    before = __reduce_add_sync(0xffffffffu, before);
    return before + sum - v;
}

// Sum of a warp's v over the warps before this one.
__device__ __forceinline__ int warp_sum_before(int v, int *warp_sums)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();  // the last call's sums have been read
    if (lane == 0) warp_sums[warp] = v;
    __syncthreads();
    return __reduce_add_sync(0xffffffffu, lane < warp ? warp_sums[lane] : 0);
}

// One moved row, by eight lanes (`lane`); 16-bit pieces, as two tokens share each
// word of the V codes and steps.
//
// What moving costs is latency: a turn is a chain of list, block table and page,
// with nothing asked for ahead.  Neither HBM (29 % of its peak) nor the issue slots
// (48 %) are full.  A pair of tokens' V is D contiguous bytes, at D = 128 four
// sectors, and each of a lane's G two-byte loads and stores touches them all again.
// 64 requests x 8 KV heads, 1.9 to 4.1 k -> 2000 slots, D = 128: 62 us with the
// finding, in 1.7 waves of blocks (64 registers at 512 threads leave two an SM).
// Moved by a second kernel, 3000 -> 2000 slots took 61 us, of which finding them 19;
// with two rows a thread at once 70, with 32 or 56 registers a thread instead of 48
// 63 to 67.
__device__ __forceinline__ void move_row(const EvictParams &p, const int32_t *table, int h, int dst, int src, int lane)
{
    const int G = p.page.groups();
    const int db = table[dst / p.page.B], sb = table[src / p.page.B];
    if (db < 0 || db >= p.num_blocks || sb < 0 || sb >= p.num_blocks) {
        if (lane == 0) record_status(p.status, KVI_ERR_OUT_OF_RANGE);
        return;
    }
    uint8_t *to = p.pool + ((int64_t)db * p.H + h) * p.page.bytes();
    const uint8_t *fr = p.pool + ((int64_t)sb * p.H + h) * p.page.bytes();
    const int d = dst % p.page.B, s = src % p.page.B;
    constexpr int kMost = KVI_MAX_ATTN_HEAD_DIM / 32;
    uint32_t k[kMost / 2];
    uint16_t v[kMost], ks = 0, vs = 0;
#pragma unroll
    for (int g = 0; g < kMost; ++g) {
        const int word = lane + 8 * g;  // of the row's 4 G words of K codes
        if (g < kMost / 2 && word < 4 * G) k[g] = *reinterpret_cast<const uint32_t *>(fr + (int64_t)s * (p.page.D / 2) + 4 * word);
        if (g < G) v[g] = *reinterpret_cast<const uint16_t *>(fr + v_piece(p.page, s, g, lane));
    }
    if (lane < G) {
        ks = *reinterpret_cast<const uint16_t *>(fr + k_step_at(p.page, s, lane));
        vs = *reinterpret_cast<const uint16_t *>(fr + v_step_at(p.page, s, lane));
    }
#pragma unroll
    for (int g = 0; g < kMost; ++g) {
        const int word = lane + 8 * g;
        if (g < kMost / 2 && word < 4 * G) *reinterpret_cast<uint32_t *>(to + (int64_t)d * (p.page.D / 2) + 4 * word) = k[g];
        if (g < G) *reinterpret_cast<uint16_t *>(to + v_piece(p.page, d, g, lane)) = v[g];
    }
    if (lane < G) {
        *reinterpret_cast<uint16_t *>(to + k_step_at(p.page, d, lane)) = ks;
        *reinterpret_cast<uint16_t *>(to + v_step_at(p.page, d, lane)) = vs;
    }
}

// ITEMS > 0: a row of at most THREADS * ITEMS slots, each read once and kept in
// registers; 0: a longer one, its ranks in shared memory (the first p.cap) and
// recomputed past them.  A warp's slots are a run of consecutive ones either way.
template <int THREADS, int ITEMS>
__global__ void __launch_bounds__(THREADS) evict_select_kernel(const __grid_constant__ EvictParams p)
{
    extern __shared__ uint32_t s_rank[];
    __shared__ int s_warp[32];
    __shared__ int s_hist[kBins];
    __shared__ int s_newest, s_digit, s_left;
    constexpr int kKept = ITEMS > 0 ? ITEMS : 1;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.x % p.H, r = blockIdx.x / p.H;
    const int64_t row = (int64_t)blockIdx.x;
    const float *w = p.w + row * p.stride;
    const int32_t *pos = p.pos + row * p.stride;
    float *w_out = p.w_out + row * p.stride;
    int32_t *pos_out = p.pos_out + row * p.stride;
    if (tid == 0) s_newest = INT32_MIN;
    for (int i = tid; i < kBins; i += THREADS) s_hist[i] = 0;
    pdl_wait();
    pdl_launch_dependents();
    const int n = p.ctx_lens[r];
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
        for (int i = tid; i < n; i += THREADS) {
            w_out[i] = w[i];
            pos_out[i] = pos[i];
        }
        if (tid == 0) p.moves[row] = 0;
        return;
    }
    const int run = ITEMS > 0 ? ITEMS * 32 : ((n + THREADS - 1) / THREADS) * 32;
    const int i0 = warp * run, i1 = min(n, i0 + run);
    float kw[kKept];
    int kp[kKept];
    uint32_t kr[kKept];
    int newest = INT32_MIN;
    if constexpr (ITEMS > 0) {
#pragma unroll
        for (int e = 0; e < ITEMS; ++e) {
            const int i = i0 + 32 * e + lane;
            kw[e] = i < i1 ? w[i] : 0.f;
            kp[e] = i < i1 ? pos[i] : INT32_MIN;
        }
#pragma unroll
        for (int e = 0; e < ITEMS; ++e) newest = max(newest, kp[e]);
    } else {
#pragma unroll 8
        for (int i = i0 + lane; i < i1; i += 32) newest = max(newest, pos[i]);
    }
    newest = __reduce_max_sync(0xffffffffu, newest);
    __syncthreads();
    if (lane == 0) atomicMax(&s_newest, newest);
    __syncthreads();
    const int64_t from = (int64_t)s_newest - p.recent + 1;
    if constexpr (ITEMS > 0) {
#pragma unroll
        for (int e = 0; e < ITEMS; ++e) kr[e] = evict_rank(kw[e], kp[e], p.sink, from);
    } else {
#pragma unroll 4
        for (int i = i0 + lane; i < i1; i += 32)
            if (i < p.cap) s_rank[i] = evict_rank(w[i], pos[i], p.sink, from);
        __syncwarp();
    }
    // f(slot, rank) for each of the warp's slots, 32 at a time and in order
    auto each = [&](auto &&f) {
        if constexpr (ITEMS > 0) {
#pragma unroll
            for (int e = 0; e < ITEMS; ++e) f(e, i0 + 32 * e + lane, kr[e]);
        } else {
            for (int i = i0; i < i1; i += 32) {
                const int at = i + lane;
                f(0, at, at >= i1 ? 0u : at < p.cap ? s_rank[at] : evict_rank(w[at], pos[at], p.sink, from));
            }
        }
    };

    // the budget-th largest rank, 11, 11 and 10 bits at a time from the top
    uint32_t found = 0;
    int want = p.budget;  // of the slots that share the bits found so far
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t mask = pass == 2 ? 1023u : 2047u;
        each([&](int, int i, uint32_t k) {
            if (i < i1 && (pass == 0 || (k ^ found) >> (pass == 1 ? 21 : 10) == 0)) atomicAdd(&s_hist[(k >> shift) & mask], 1);
        });
        __syncthreads();
        // from the top bin down, a few bins a thread: the one where the count
        // passes `want`
        constexpr int kOwn = kBins / THREADS;
        const int hi = kBins - 1 - kOwn * tid;
        int count[kOwn], all = 0;
#pragma unroll
        for (int e = 0; e < kOwn; ++e) {
            count[e] = s_hist[hi - e];
            s_hist[hi - e] = 0;
            all += count[e];
        }
        int above = block_sum_before(all, s_warp);
#pragma unroll
        for (int e = 0; e < kOwn; ++e) {
            if (above < want && above + count[e] >= want) {
                s_digit = hi - e;
                s_left = want - above;
            }
            above += count[e];
        }
        __syncthreads();
        found |= (uint32_t)s_digit << shift;
        want = s_left;
    }
    // ranks above `found` stay, and the first `want` slots that equal it; each
    // warp counts its run, and then knows its places in the lists
    const uint32_t below = (1u << lane) - 1u;
    int32_t *holes = p.holes + row * p.most, *tails = p.tails + row * p.most;
    int ties = 0;
    each([&](int, int i, uint32_t k) { ties += __popc(__ballot_sync(0xffffffffu, i < i1 && k == found)); });
    const int ties0 = warp_sum_before(ties, s_warp);
    int hole_at = 0, tail_at = 0;
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
        int tie_at = ties0;
        each([&](int e, int i, uint32_t k) {
            const bool in = i < i1;
            const uint32_t tie = __ballot_sync(0xffffffffu, in && k == found);
            const bool keep = in && (k > found || (k == found && tie_at + __popc(tie & below) < want));
            tie_at += __popc(tie);
            const bool hole = in && i < left && !keep, tail = keep && i >= left;
            const uint32_t hs = __ballot_sync(0xffffffffu, hole), ts = __ballot_sync(0xffffffffu, tail);
            if (pass == 1) {
                if (hole) holes[hole_at + __popc(hs & below)] = i;
                if (tail) tails[tail_at + __popc(ts & below)] = i;
                if (in && !hole) {
                    w_out[i] = i >= left ? 0.f : ITEMS > 0 ? kw[e] : w[i];
                    pos_out[i] = i >= left ? -1 : ITEMS > 0 ? kp[e] : pos[i];
                }
            }
            hole_at += __popc(hs);
            tail_at += __popc(ts);
        });
        if (pass == 0) {
            hole_at = warp_sum_before(hole_at, s_warp);
            tail_at = warp_sum_before(tail_at, s_warp);
        } else if (tid == THREADS - 1) {
            s_left = hole_at;  // all of them
        }
    }
    __syncthreads();
    const int n_holes = s_left;
#pragma unroll 2
    for (int i = tid; i < n_holes; i += THREADS) {
        const int to = holes[i], at = tails[i];
        w_out[to] = w[at];
        pos_out[to] = pos[at];
    }
    if (p.move_here) {
        const int32_t *table = p.block_tables + (int64_t)r * p.max_blocks;
        for (int i = tid >> 3; i < n_holes; i += THREADS / 8) move_row(p, table, h, holes[i], tails[i], tid & 7);
    } else if (tid == 0) {
        p.moves[row] = n_holes;
    }
}

// The rows of few heads that have many each.
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ EvictParams p)
{
    pdl_wait();
    pdl_launch_dependents();
    const int64_t row = blockIdx.y;
    const int h = (int)(row % p.H), r = (int)(row / p.H);
    const int i = blockIdx.x * (kMoveThreads / 8) + (threadIdx.x >> 3);
    if (i >= p.moves[row]) return;
    move_row(p, p.block_tables + (int64_t)r * p.max_blocks, h, p.holes[row * p.most + i], p.tails[row * p.most + i],
             threadIdx.x & 7);
}

// A block's threads and the slots a thread keeps, by the longest row.
cudaError_t launch_select(EvictParams &p, unsigned rows, cudaStream_t s)
{
    if (p.max_ctx <= 2048) return launch_chained(evict_select_kernel<512, 4>, dim3(rows), 512, 0, s, p);
    if (p.max_ctx <= 4096) return launch_chained(evict_select_kernel<512, 8>, dim3(rows), 512, 0, s, p);
    if (p.max_ctx <= 8192) return launch_chained(evict_select_kernel<1024, 8>, dim3(rows), 1024, 0, s, p);
    p.cap = std::min(p.max_ctx, kRankCap);
    const cudaError_t e = smem_opt_in(evict_select_kernel<1024, 0>, kRankCap * 4);
    if (e != cudaSuccess) return e;
    return launch_chained(evict_select_kernel<1024, 0>, dim3(rows), 1024, (size_t)p.cap * 4, s, p);
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
    if (T >= 0xfffffff0ll) return arg_error("T=%lld rows are too many", (long long)T);
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

// A block's shape, and the grid: pairs of rows on x (one more than half the
// rows, as pairs may start at row -1), the parts of a wide pair on y.
void row_shape(RowParams &p, dim3 &grid, dim3 &block)
{
    // a head a thread while that keeps the threads below a wave of them, else
    // four, which share a thread's looking up and addressing (stored and read back,
    // 8 heads of 128 channels: 65 k rows 145 us with one head a thread, 123 with two,
    // 117 with four, 153 with eight; 64 rows 5.5 us with one, 13 with four)
    const int64_t threads = (p.T / 2 + 1) * p.H * (p.D / 8);
    p.heads_apart = threads <= (int64_t)kPlanSms * 2048 ? p.H : (p.H + 3) / 4;
    p.lanes = p.heads_apart * (p.D / 8);  // a multiple of 4: a group never leaves its warp
    // whole warps: eight pairs together are one, or a pair is rounded up
    const int x = p.lanes <= 32 ? p.lanes : std::min((p.lanes + 31) & ~31, kRowThreads);
    const int y = p.lanes <= 32 ? (kRowThreads / x) & ~7 : kRowThreads / x;
    const int64_t pairs = p.T / 2 + 1;
    block = dim3((unsigned)x, (unsigned)y);
    grid = dim3((unsigned)((pairs + y - 1) / y), (unsigned)((p.lanes + x - 1) / x));
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
    dim3 grid, block;
    row_shape(p, grid, block);
    return cuda_status(launch_chained(cache4_write_kernel, grid, block, 0, stream, p), "kvi_cache4_write");
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
    dim3 grid, block;
    row_shape(p, grid, block);
    return cuda_status(launch_chained(cache4_read_kernel, grid, block, 0, stream, p), "kvi_cache4_read");
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
    const int rows = std::min(budget, max_ctx - budget);  // a head moves at most so many
    // Moved by the block that found them where those are few, or the blocks many:
    // 8 KV heads, 1 request: 101 rows a head 7.5 us so, 7.9 by a second kernel;
    // 577 rows 11.4 and 7.9; 16 requests, 800 rows: 12.4 and 15.4 (4: 11.8, 10.9).
    p.move_here = rows <= 128 || (int64_t)R * kv_heads >= 128;
    cudaError_t e = launch_select(p, (unsigned)(R * kv_heads), stream);
    st = cuda_status(e, "kvi_cache4_evict");
    if (st != KVI_OK || rows <= 0 || p.move_here) return st;
    const unsigned gx = (unsigned)((rows + kMoveThreads / 8 - 1) / (kMoveThreads / 8));
    const dim3 grid(gx, (unsigned)(R * kv_heads));
    e = launch_chained(evict_move_kernel, grid, kMoveThreads, 0, stream, p);
    return cuda_status(e, "kvi_cache4_evict");
}
