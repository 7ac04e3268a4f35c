// kvi_attn_decode4.cu -- one decoding step over the 4-bit cache.
//
// For each request and query head: s_p = scale <q, k_p>, out = sum softmax(s)_p
// v_p over the cached keys, k = step * code and v likewise.  The cache is read
// once and nothing else is large, so HBM bounds it: D + D / 8 bytes per key
// and KV head.
//
// Tensor cores with the keys on M.  Few rows of q read each key (the heads of
// its group), so the products are taken as S^T = K Q^T (16 keys x 8 heads)
// and O^T = V^T P^T (16 channels x 8 heads): up to 8 heads fill N without
// padding, half of what heads on M = 16 would pad to.  The page layout is
// this instruction's fragment order, so a lane reads its share of 16 tokens
// with a few wide loads.
//   K: a group's product is taken of the bare codes and then scaled by the
//      key's step in float32 (step * code has 12 significant bits and would
//      not fit a bf16 operand).
//   V: the step belongs to (key, group), and a key is summed over, so it is P
//      that is scaled; P * step rounds to bf16, as any P on tensor cores does.
//   A nibble c of a 16-bit half, or'ed with 0x4300, is the bf16 number 128 + c
//      if it is the lowest; or'ed with 0x6400, the f16 number 1024 + c if it is
//      the lowest and 1024 + 16 c if it is the next.  136, or 1032, or 64 + 8
//      after a division by 16, is subtracted exactly.  K is taken in f16, which
//      needs half the shifts; V in bf16, as P * step has no bound that fits f16.
// A warp takes pairs of tiles of 16 keys in turn, from a ring of its own that
// bulk copies fill ahead of it, with a softmax of its own; the warps of a block
// join at the end, and blocks that share a request's keys through one another's
// shared memory as a cluster, or in a second kernel.
//
// What bounds it is the decoding, not the bytes: with the softmax a tile of 2304
// bytes (D = 128) takes nearly 400 warp instructions, and HBM delivers a tile in
// the time of 390.  128 registers leave 16 warps an SM, four a scheduler, and an
// iteration is a chain (scores, softmax, weights, output): two thirds of the issue
// slots are used, the rest goes into its fixed latencies and the ALU pipe (59 %).  Measured at 16 requests x 28 k keys, D = 128, 8 KV heads (0.53
// GB): 125 us, 4.2 TB/s.  On the way there: one tile an iteration 152 us; two,
// which share the bookkeeping and run independently of one another, 140, later
// 132; K in f16 129; more and shorter pieces 125.  Against the 140:
// 12 warps an SM instead of 16 took 148, shifts as multiplications 166, the
// offset of V's codes taken off by a second matrix product 155.
#include <cuda_runtime.h>

#include <algorithm>

#include "kvi_attn.cuh"
#include "kvi_sync.cuh"

namespace kvi {

namespace {

constexpr int kWarps4 = 4;
constexpr int kStages4 = 2;  // pairs of tiles of 16 keys that a warp has in flight
constexpr uint64_t kWait4Ns = 1000000000ull;

struct Decode4Params {
    const __nv_bfloat16 *q;
    int64_t q_stride;
    const int32_t *ctx_lens;
    int32_t max_ctx, max_blocks;
    const int32_t *block_tables;
    int32_t num_blocks;
    int32_t H, Hq, G;
    int32_t chunks;  // of 8 * NT heads each that a group takes
    Page4 page;
    const uint8_t *pool;
    float scale;     // times log2 e
    __nv_bfloat16 *out;
    int64_t out_stride;
    int32_t S, span;
    int32_t joined;  // a request's pieces are a cluster, which joins them
    float *po;
    float2 *ml;
    float *scores;   // [R][H][max_ctx][score_stride] or null
    int32_t score_stride;
    int32_t *status;
};

// N 32-bit words from shared memory, with the widest loads their count allows
// (p is aligned to that width).
template <int N>
__device__ __forceinline__ void load_words(uint32_t (&w)[N], const uint8_t *p)
{
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const uint4 v = reinterpret_cast<const uint4 *>(p)[i];
            w[4 * i] = v.x;
            w[4 * i + 1] = v.y;
            w[4 * i + 2] = v.z;
            w[4 * i + 3] = v.w;
        }
    } else if constexpr (N % 2 == 0) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const uint2 v = reinterpret_cast<const uint2 *>(p)[i];
            w[2 * i] = v.x;
            w[2 * i + 1] = v.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = reinterpret_cast<const uint32_t *>(p)[i];
    }
}

// N bf16 numbers from p, packed two to a word.
template <int N>
__device__ __forceinline__ void load_halves(uint32_t (&w)[(N + 1) / 2], const uint8_t *p)
{
    if constexpr (N % 2 == 0) {
        load_words<N / 2>(w, p);
    } else {
        const uint16_t *h = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
        for (int i = 0; i < (N + 1) / 2; ++i)
            w[i] = (uint32_t)h[2 * i] | (2 * i + 1 < N ? (uint32_t)h[2 * i + 1] << 16 : 0u);
    }
}

__device__ __forceinline__ void bulk_copy(uint32_t dst, const uint8_t *src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// Shared memory of a block: each warp's ring of stages, two tiles of 16 tokens
// each (a tile in the order of a page of 16 tokens: K codes, V codes, K steps,
// V steps), reused for the join.
template <int NG, int NT>
struct Smem4 {
    static constexpr int kCodes = 256 * NG, kSteps = 32 * NG;
    static constexpr int kTile = 2 * kCodes + 2 * kSteps;
    static constexpr int kStage = 2 * kTile;
    static constexpr int kRing = kStages4 * kStage;
    static constexpr int kSum = kWarps4 * 8 * NT * (32 * NG + 4) * 4;  // then the block's own
    static constexpr int kJoin = kSum + 8 * NT * 32 * NG * 4;
    static constexpr int kBytes = kWarps4 * kRing > kJoin ? kWarps4 * kRing : kJoin;
};

// JOINED: a request's pieces are a cluster, which joins them.  (A kernel of its
// own, as the join's registers are the loop's: 16 x 28 k keys 128 us in one, 125.)
template <int NG, int NT, bool JOINED>
__global__ void __launch_bounds__(kWarps4 * 32, NG * NT <= 4 ? 4 : NG * NT <= 6 ? 3 : 2)
decode4_kernel(const __grid_constant__ Decode4Params p)
{
    using Sm = Smem4<NG, NT>;
    constexpr int D = NG * 32;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t s_bar[kWarps4][kStages4];
    __shared__ float s_m[kWarps4][8 * NT], s_l[kWarps4][8 * NT];
    __shared__ float2 s_ml[8 * NT];  // of the block
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int split = blockIdx.x;
    const int h = blockIdx.y / p.chunks, c0 = (blockIdx.y % p.chunks) * 8 * NT;  // first head of the group
    const int r = blockIdx.z;
    pdl_wait();
    pdl_launch_dependents();
    RequestSpan rq;
    if (!request_span(r, nullptr, (int)gridDim.z, 1, p.ctx_lens, p.max_ctx, p.max_blocks, p.page.B, rq)) {
        if (tid == 0) record_status(p.status, KVI_ERR_OUT_OF_RANGE);
        return;
    }
    const int from = split * p.span, to = min(rq.ctx, from + p.span);
    const bool whole = rq.ctx <= p.span;
    if (from >= to && split > 0) {  // split 0 writes the zeros of an empty cache
        if (JOINED && !whole) {  // (the others of the cluster count on it)
            cluster_sync();
            cluster_sync();
        }
        return;
    }

    // ---- this warp's pairs of tiles: from / 32 + warp, + kWarps4, ...; a stage each
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < kStages4; ++i) mbar_init(smem_u32(&s_bar[warp][i]), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
    uint8_t *ring = smem + warp * Sm::kRing;
    const int32_t *table = p.block_tables + (int64_t)r * p.max_blocks;
    const int t1 = (to + 15) / 16, pair0 = from / 32 + warp;
    const int per_page = p.page.B / 16;
    const int64_t page_bytes = p.page.bytes(), block_bytes = page_bytes * p.H;
    // The copies of a stage, one lane each: lane % 4 is the part of the tile
    // (K codes, V codes, K steps, V steps; a page of 16 tokens is one part) and
    // lane / 4 the tile.  Each lane keeps its next tile's place in the table and in
    // its page, stepped by a division made once, and reads the tile's block
    // an iteration ahead, so that the two latencies do not add up.
    const int part = lane & 3;
    const bool copies = lane < 8 && (part == 0 || per_page > 1);
    const uint32_t part_bytes = per_page == 1 ? Sm::kTile : part < 2 ? Sm::kCodes : Sm::kSteps;
    const uint32_t part_dst = smem_u32(ring) + ((lane >> 2) & 1) * Sm::kTile +
                              (part < 2 ? part * Sm::kCodes : 2 * Sm::kCodes + (part - 2) * Sm::kSteps);
    const uint8_t *part_src = p.pool + h * page_bytes +
                              (part == 0 ? 0 : part == 1 ? p.page.v_codes() : part == 2 ? p.page.k_steps() : p.page.v_steps());
    int c_tile = 2 * pair0 + ((lane >> 2) & 1), c_page = c_tile / per_page, c_sub = c_tile % per_page;
    const int d_page = 2 * kWarps4 / per_page, d_sub = 2 * kWarps4 % per_page;
    int c_block = c_tile < t1 ? table[c_page] : -1;
    int issued = 0;     // stages that copies went out for
    uint32_t dead = 0;  // bits 2 stage, + 1: a tile whose block lies outside the pool
    auto issue = [&](int stage) {
        // a tile past the end is not copied: its keys are masked
        const bool live = (uint32_t)c_block < (uint32_t)p.num_blocks;
        const uint32_t lives = __ballot_sync(0xffffffffu, live) & 0x11u;
        const uint32_t bar = smem_u32(&s_bar[warp][stage]);
        if (lives != 0x11u) {
            const uint32_t lost = __ballot_sync(0xffffffffu, !live && c_tile < t1) & 0x11u;
            if (lost && lane == 0) record_status(p.status, KVI_ERR_OUT_OF_RANGE);
            dead = (dead & ~(3u << (2 * stage))) | (((lost & 1u) | (lost >> 3)) << (2 * stage));
        } else if (dead) {
            dead &= ~(3u << (2 * stage));
        }
        if (lane == 0) mbar_expect_tx(bar, __popc(lives) * Sm::kTile);
        __syncwarp();
        if (copies && live)
            bulk_copy(part_dst + stage * Sm::kStage, part_src + c_block * block_bytes + c_sub * part_bytes, part_bytes, bar);
        ++issued;
        c_tile += 2 * kWarps4;
        c_page += d_page;
        c_sub += d_sub;
        if (c_sub >= per_page) {
            c_sub -= per_page;
            ++c_page;
        }
        c_block = c_tile < t1 ? table[c_page] : -1;
    };
    const int pairs = max(0, ((t1 + 1) / 2 - pair0 + kWarps4 - 1) / kWarps4);  // of this warp
#pragma unroll
    for (int i = 0; i < kStages4; ++i)
        if (i < pairs) issue(i);

    // Q as B fragments: word (a, b) of group j is channels 32 j + 8 t + 2 a + b
    // and + 4, the order of the codes' nibbles.  In f16, each head scaled by a power
    // of two that brings its largest element to 2^13: f16 keeps three more bits
    // than bf16 has, and what it loses of elements below 2^-27 of the largest is
    // nothing beside float32 sums.  The scale of the scores takes it back.
    uint32_t qf[NT][2 * NG][2];
    float scale[NT][2];  // of columns (heads) 2 t and 2 t + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int head = c0 + 8 * nt + g;
        const __nv_bfloat16 *q = p.q + (int64_t)r * p.q_stride + ((int64_t)h * p.G + head) * D + 8 * t;
        uint4 v[NG];
        uint32_t top = 0;  // the largest |q| as bf16 bits
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            v[j] = make_uint4(0, 0, 0, 0);
            if (head < p.G) v[j] = *reinterpret_cast<const uint4 *>(q + 32 * j);
            const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^(13 - e) and 2^(e - 13) of a largest element in [2^e, 2^(e + 1)); both are
        // normal numbers for any finite q (an infinity or NaN stays one), and heads
        // below 2^-100 are taken as if they reached it, for kLazy / scale
        const int e = min(max((int)(top >> 7) - 127, -100), 127);
        const float up = __int_as_float((127 + 13 - e) << 23), down = __int_as_float((127 - 13 + e) << 23);
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            // v = channels (0,1) (2,3) (4,5) (6,7)
            qf[nt][2 * j][0] = pack_f16(bf16_lo(v[j].x) * up, bf16_lo(v[j].z) * up);      // 0, 4
            qf[nt][2 * j][1] = pack_f16(bf16_hi(v[j].x) * up, bf16_hi(v[j].z) * up);      // 1, 5
            qf[nt][2 * j + 1][0] = pack_f16(bf16_lo(v[j].y) * up, bf16_lo(v[j].w) * up);  // 2, 6
            qf[nt][2 * j + 1][1] = pack_f16(bf16_hi(v[j].y) * up, bf16_hi(v[j].w) * up);  // 3, 7
        }
#pragma unroll
        for (int c = 0; c < 2; ++c)  // (never 0, or a masked score would be NaN: 0 * inf)
            scale[nt][c] = fmaxf(p.scale * __shfl_sync(0xffffffffu, down, 4 * (2 * t + c)), 1.1754944e-38f);
    }
    float o[NT][2 * NG][4];
    // per column (head): the score that moves the reference (-inf while there is
    // none), the reference as an exponent, and this lane's share of the sum
    float limit[NT][2], ref[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < 2 * NG; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[nt][i][j] = 0.f;
        limit[nt][0] = limit[nt][1] = neg_inf();
        ref[nt][0] = ref[nt][1] = l[nt][0] = l[nt][1] = 0.f;
    }

    int stage = 0;
    uint32_t phase = 0;
    for (int it = 0; it < pairs; ++it) {
        // (agreed on: what follows wants the whole warp, and a lane alone could give up
        // where the others find the copy there)
        if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&s_bar[warp][stage]), phase, kWait4Ns))) {
            record_status(p.status, KVI_ERR_TIMEOUT);
            break;
        }
        const uint8_t *st = ring + stage * Sm::kStage;
        const int k0 = (pair0 + it * kWarps4) * 32;  // the pair's first key
        const uint32_t lost = dead >> (2 * stage);
        const bool partly = k0 + 32 > to || (lost & 3u);
        // keys of tile f: there are those below `to`, unless the tile is lost
        const int end[2] = {lost & 1u ? 0 : to, lost & 2u ? 0 : to};
        // ---- scores: keys g and g + 8 of each tile, heads 2 t and 2 t + 1
        float s[2][NT][4];
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            uint32_t kc[2][NG], ks[2][(NG + 1) / 2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                load_words<NG>(kc[i], st + f * Sm::kTile + (g + 8 * i) * (NG * 16) + t * (NG * 4));
                load_halves<NG>(ks[i], st + f * Sm::kTile + 2 * Sm::kCodes + (g + 8 * i) * (NG * 2));
            }
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                const float s0 = (j & 1) ? bf16_hi(ks[0][j / 2]) : bf16_lo(ks[0][j / 2]);
                const float s1 = (j & 1) ? bf16_hi(ks[1][j / 2]) : bf16_lo(ks[1][j / 2]);
                float sum[NT][4];
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    const uint32_t x = kc[0][j] >> (8 * a), y = kc[1][j] >> (8 * a);
                    const uint32_t a0 = codes_f16x2(x), a1 = codes_f16x2(y), a2 = codes_f16x2_high(x), a3 = codes_f16x2_high(y);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        if (a == 0)
                            mma16816_f16_first(sum[nt], a0, a1, a2, a3, qf[nt][2 * j][0], qf[nt][2 * j][1]);
                        else
                            mma16816_f16(sum[nt], a0, a1, a2, a3, qf[nt][2 * j + 1][0], qf[nt][2 * j + 1][1]);
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        s[f][nt][i] = j ? fmaf(i < 2 ? s0 : s1, sum[nt][i], s[f][nt][i]) : (i < 2 ? s0 : s1) * sum[nt][i];
            }
        }
        if (partly) {
#pragma unroll
            for (int f = 0; f < 2; ++f)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (k0 + 16 * f + g + (i >> 1) * 8 >= end[f]) s[f][nt][i] = neg_inf();
        }
        bool move = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c)
                move |= fmaxf(fmaxf(s[0][nt][c], s[0][nt][c + 2]), fmaxf(s[1][nt][c], s[1][nt][c + 2])) > limit[nt][c];
        if (p.scores) {
#pragma unroll
            for (int f = 0; f < 2; ++f)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const int head = c0 + 8 * nt + 2 * t, key = k0 + 16 * f + g;
                    float *sc = p.scores + (((int64_t)r * p.H + h) * p.max_ctx + key) * p.score_stride + head;
                    if (head < p.score_stride) {
                        if (key < to)
                            *reinterpret_cast<float2 *>(sc) = make_float2(s[f][nt][0] * scale[nt][0], s[f][nt][1] * scale[nt][1]);
                        if (key + 8 < to)
                            *reinterpret_cast<float2 *>(sc + 8 * p.score_stride) =
                                make_float2(s[f][nt][2] * scale[nt][0], s[f][nt][3] * scale[nt][1]);
                    }
                }
        }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float top = fmaxf(fmaxf(s[0][nt][c], s[0][nt][c + 2]), fmaxf(s[1][nt][c], s[1][nt][c + 2]));
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                    // each column goes by its own scores alone
                    if (!(top > limit[nt][c])) continue;
                    const float to = top * scale[nt][c];
                    const float f = limit[nt][c] == neg_inf() ? 0.f : exp2_fast(ref[nt][c] - to);
                    limit[nt][c] = top + kLazy / scale[nt][c];
                    ref[nt][c] = to;
                    l[nt][c] *= f;
#pragma unroll
                    for (int i = 0; i < 2 * NG; ++i) {
                        o[nt][i][c] *= f;
                        o[nt][i][c + 2] *= f;
                    }
                }
            __syncwarp();  // the next matrix instruction wants the warp as one
        }
        // ---- weights, as B fragments: keys 2 t, 2 t + 1 (and + 8) of head g,
        // in two parts, P = hi + lo, so that P * step rounds to bf16 once
        uint32_t b0[2][NT], b1[2][NT], r0[2][NT], r1[2][NT];
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float p0 = exp2_fast(fmaf(s[f][nt][0], scale[nt][0], -ref[nt][0]));
                const float p1 = exp2_fast(fmaf(s[f][nt][1], scale[nt][1], -ref[nt][1]));
                const float p2 = exp2_fast(fmaf(s[f][nt][2], scale[nt][0], -ref[nt][0]));
                const float p3 = exp2_fast(fmaf(s[f][nt][3], scale[nt][1], -ref[nt][1]));
                l[nt][0] += p0 + p2;
                l[nt][1] += p1 + p3;
                const uint32_t h0 = pack_bf16(p0, p1), h1 = pack_bf16(p2, p3);
                b0[f][nt] = transpose8x8(h0);
                b1[f][nt] = transpose8x8(h1);
                r0[f][nt] = transpose8x8(pack_bf16(p0 - bf16_lo(h0), p1 - bf16_hi(h0)));
                r1[f][nt] = transpose8x8(pack_bf16(p2 - bf16_lo(h1), p3 - bf16_hi(h1)));
            }
        // ---- output: channels 32 j + 4 g + 2 a (+ 1), heads 2 t and 2 t + 1
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            uint32_t vc[2][NG], vs[2][NG];  // token pairs t and t + 4
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                load_words<NG>(vc[i], st + f * Sm::kTile + Sm::kCodes + (t + 4 * i) * (NG * 32) + g * (NG * 4));
                load_words<NG>(vs[i], st + f * Sm::kTile + 2 * Sm::kCodes + Sm::kSteps + (t + 4 * i) * (NG * 4));
            }
            // slots past the end have weight 0, but their steps may hold anything
            if (partly) {
                const int k = k0 + 16 * f + 2 * t;
                const uint32_t keep0 = (k < end[f] ? 0x0000ffffu : 0u) | (k + 1 < end[f] ? 0xffff0000u : 0u);
                const uint32_t keep1 = (k + 8 < end[f] ? 0x0000ffffu : 0u) | (k + 9 < end[f] ? 0xffff0000u : 0u);
#pragma unroll
                for (int j = 0; j < NG; ++j) {
                    vs[0][j] &= keep0;
                    vs[1][j] &= keep1;
                }
            }
            if (f == 1) {
                __syncwarp();  // the stage is in registers
                if (it + kStages4 < pairs) issue(stage);
            }
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                uint32_t w0[NT], w1[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    w0[nt] = scale_bf16x2(b0[f][nt], r0[f][nt], vs[0][j]);
                    w1[nt] = scale_bf16x2(b1[f][nt], r1[f][nt], vs[1][j]);
                }
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    const uint32_t a0 = codes_bf16x2(vc[0][j] >> (8 * a)), a1 = codes_bf16x2(vc[0][j] >> (8 * a + 4));
                    const uint32_t a2 = codes_bf16x2(vc[1][j] >> (8 * a)), a3 = codes_bf16x2(vc[1][j] >> (8 * a + 4));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma16816(o[nt][2 * j + a], a0, a1, a2, a3, w0[nt], w1[nt]);
                }
            }
        }
        if (++stage == kStages4) {
            stage = 0;
            phase ^= 1u;
        }
    }
    // after a wait that gave up: no copy may still be writing when the rings
    // are reused (bounded; the outputs are not valid, as the status says)
    if (lane < kStages4 && lane < issued) {
        const int last = (issued - 1 - lane) / kStages4;
        if (!mbar_wait(smem_u32(&s_bar[warp][lane]), (uint32_t)(last & 1), kWait4Ns))
            record_status(p.status, KVI_ERR_TIMEOUT);
    }
    __syncthreads();
    float *s_o = reinterpret_cast<float *>(smem);
    constexpr int kO = D + 4;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], off);
            const int n = 8 * nt + 2 * t + c;
            if (g == 0) {
                s_m[warp][n] = limit[nt][c] == neg_inf() ? neg_inf() : ref[nt][c];
                s_l[warp][n] = l[nt][c];
            }
#pragma unroll
            for (int j = 0; j < NG; ++j)
                *reinterpret_cast<float4 *>(s_o + (warp * 8 * NT + n) * kO + 32 * j + 4 * g) =
                    make_float4(o[nt][2 * j][c], o[nt][2 * j][c + 2], o[nt][2 * j + 1][c], o[nt][2 * j + 1][c + 2]);
        }
    }
    __syncthreads();
    for (int i = tid; i < 8 * NT * (D / 2); i += kWarps4 * 32) {
        const int n = i / (D / 2), d = (i % (D / 2)) * 2;
        if (c0 + n >= p.G) continue;
        float M = neg_inf();
#pragma unroll
        for (int w = 0; w < kWarps4; ++w) M = fmaxf(M, s_m[w][n]);
        const float ref = M == neg_inf() ? 0.f : M;
        float L = 0.f;
        float2 acc = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps4; ++w) {
            const float f = exp2_fast(s_m[w][n] - ref);
            L += s_l[w][n] * f;
            const float *src = s_o + (w * 8 * NT + n) * kO + d;
            acc.x += src[0] * f;
            acc.y += src[1] * f;
        }
        const int64_t row = (int64_t)r * p.Hq + (int64_t)h * p.G + c0 + n;
        if (whole) {
            const float inv = L == 0.f ? 0.f : 1.f / L;
            *reinterpret_cast<uint32_t *>(p.out + (int64_t)r * p.out_stride + ((int64_t)h * p.G + c0 + n) * D + d) =
                pack_bf16(acc.x * inv, acc.y * inv);
        } else if (JOINED) {
            *reinterpret_cast<float2 *>(smem + Sm::kSum + (n * D + d) * 4) = acc;
            if (d == 0) s_ml[n] = make_float2(M, L);
        } else {
            *reinterpret_cast<float2 *>(p.po + (row * p.S + split) * D + d) = acc;
        }
        if (!JOINED && d == 0 && (!whole || p.scores)) p.ml[row * p.S + split] = make_float2(M, L);
    }
    if (!JOINED || whole) return;
    // ---- each block of the cluster that has keys joins a part of the channels
    cluster_sync();
    const int pieces = (rq.ctx + p.span - 1) / p.span;
    for (int i = split * kWarps4 * 32 + tid; i < 8 * NT * (D / 2); i += pieces * kWarps4 * 32) {
        const int n = i / (D / 2), d = (i % (D / 2)) * 2;
        if (c0 + n >= p.G) continue;
        float2 ml[kMostJoined], part[kMostJoined];
        float M = neg_inf();
#pragma unroll
        for (int k = 0; k < kMostJoined; ++k) {
            if (k >= pieces) continue;
            ml[k] = load_of_block(smem_u32(&s_ml[n]), k);
            part[k] = load_of_block(smem_u32(smem + Sm::kSum + (n * D + d) * 4), k);
            M = fmaxf(M, ml[k].x);
        }
        const float ref = M == neg_inf() ? 0.f : M;
        float L = 0.f;
        float2 acc = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kMostJoined; ++k) {
            if (k >= pieces) continue;
            const float f = exp2_fast(ml[k].x - ref);
            L += ml[k].y * f;
            acc.x += part[k].x * f;
            acc.y += part[k].y * f;
        }
        const float inv = L == 0.f ? 0.f : 1.f / L;
        *reinterpret_cast<uint32_t *>(p.out + (int64_t)r * p.out_stride + ((int64_t)h * p.G + c0 + n) * D + d) =
            pack_bf16(acc.x * inv, acc.y * inv);
    }
    cluster_sync();  // no block leaves while its sums are read
}

// ------------------------------------------------------ accumulated weights

struct WeightParams {
    JoinParams join;
    int32_t join_blocks;  // 0: every request has a single piece
    int32_t key_blocks;   // per KV head
    const float *scores;
    int32_t score_stride;
    int32_t H, G;
    float *w;
    int64_t stride;
};

constexpr int kKeysThread = 4;
constexpr int kKeysBlock = kKeysThread * kJoinWarps * 32;

// After the attention, per request: blocks that join its pieces' outputs, and
// blocks that add weights[r][h][p] += sum over the group's heads of
// 2^(s_p - M) / L, from the scores that the attention left.
__global__ void __launch_bounds__(kJoinWarps * 32) finish_kernel(const __grid_constant__ WeightParams p)
{
    __shared__ float s_ref[KVI_MAX_ATTN_GROUP], s_inv[KVI_MAX_ATTN_GROUP];
    pdl_wait();
    pdl_launch_dependents();
    const JoinParams &jp = p.join;
    const int r = blockIdx.y, tid = threadIdx.x;
    if ((int)blockIdx.x < p.join_blocks) {
        join_rows(jp, blockIdx.x, r);
        return;
    }
    const int x = blockIdx.x - p.join_blocks, h = x / p.key_blocks;
    RequestSpan rq;
    if (!request_span(r, nullptr, jp.total_q, 1, jp.ctx_lens, jp.max_ctx, jp.max_blocks, jp.block_size, rq)) return;
    const int key0 = (x % p.key_blocks) * kKeysBlock;
    if (key0 >= rq.ctx) return;
    // the scores of a thread's keys, up to eight heads of each, are asked for before
    // the sums that they are measured against
    const float *sc = p.scores + ((int64_t)r * p.H + h) * jp.max_ctx * p.score_stride;
    float *w = p.w + ((int64_t)r * p.H + h) * p.stride;
    constexpr int kAhead = 4;
    float2 ahead[kKeysThread][kAhead];
    float old[kKeysThread];
#pragma unroll
    for (int e = 0; e < kKeysThread; ++e) {
        const int key = key0 + e * kJoinWarps * 32 + tid;
        if (key >= rq.ctx) continue;
        old[e] = w[key];
#pragma unroll
        for (int g = 0; g < kAhead; ++g)
            if (2 * g < p.G) ahead[e][g] = *reinterpret_cast<const float2 *>(sc + (int64_t)key * p.score_stride + 2 * g);
    }
    const int pieces = (rq.ctx + jp.span - 1) / jp.span;
    // a warp per head
    for (int g = tid >> 5; g < p.G; g += kJoinWarps) {
        const int lane = tid & 31;
        const float2 *ml = jp.ml + ((int64_t)r * jp.q_heads + (int64_t)h * p.G + g) * jp.S;
        float M = neg_inf();
        for (int s = lane; s < pieces; s += 32) M = fmaxf(M, ml[s].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        const float ref = M == neg_inf() ? 0.f : M;
        float L = 0.f;
        for (int s = lane; s < pieces; s += 32) L += ml[s].y * exp2_fast(ml[s].x - ref);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
        if (lane == 0) {
            s_ref[g] = ref;
            s_inv[g] = L == 0.f ? 0.f : 1.f / L;
        }
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kKeysThread; ++e) {
        const int key = key0 + e * kJoinWarps * 32 + tid;
        if (key >= rq.ctx) break;
        const float *s = sc + (int64_t)key * p.score_stride;
        float sum = 0.f;
#pragma unroll
        for (int g = 0; g < kAhead; ++g) {
            if (2 * g < p.G) sum += exp2_fast(ahead[e][g].x - s_ref[2 * g]) * s_inv[2 * g];
            if (2 * g + 1 < p.G) sum += exp2_fast(ahead[e][g].y - s_ref[2 * g + 1]) * s_inv[2 * g + 1];
        }
        for (int g = 2 * kAhead; g < p.G; ++g) sum += exp2_fast(s[g] - s_ref[g]) * s_inv[g];
        w[key] = old[e] + sum;
    }
}

// -------------------------------------------------------------------- host

struct Plan4 {
    int nt, chunks, S, span;
    bool joined;
    size_t ml, scores, total;  // byte offsets after the partial outputs
    int score_stride;
};

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// Pieces of a request's keys.  A wave is four blocks on every SM.  (us, 8 KV heads
// of 128 channels, requests x keys, by the number of pieces:)
//  - One wave where the rows divide it well and the pieces stay short, as a part
//    of a second wave costs most of a whole one: 16 x 2048 4: 15.6, 8: 17.5; 24 x
//    4096 3: 32.4, 6: 36.1; 64 x 2048 1: 39.7, 3: 46.6.
//  - Else two waves, whose ends even out: 40 x 2048 1: 36.4, 4: 30.8; and up to
//    four where the pieces are long: 16 x 28000 4: 119.7, 10: 114.2, 14: 110.3.
//    Lengths from half of max_ctx up, 24 x 8192 3: 53.0, 8: 45.2; 16 x 28000 4:
//    118.9, 10: 94.5, 14: 91.3 (24 x 2048 the same, 64 x 2048 1: 36.2, 3: 37.0).
//  - No more than 16 pieces, or one per 1024 keys, for the join reads them one
//    after the other: 1 x 8192 16: 10.6, 64: 15.1; 1 x 28000 32: 17.5, 73: 21.8.
//  - 8 instead of 9 to 16 where a cluster then joins them (below) and they stay
//    short: 4 x 4096 8: 11.4, 16: 12.2; 1 x 1601 7.5 and 7.6, 1 x 4096 9.5 and 8.6.
//  - One piece, and no join, for few keys: 1 x 384 1: 6.1, 3: 6.2; 16 x 600 1:
//    8.8, 2: 10.2; 1 x 600 1: 8.7, 5: 6.9.
constexpr int64_t kWave = 4 * kPlanSms;
constexpr int kAlone = 384, kLongest = 1 << 30;  // keys that are never split, and of a piece at most

int64_t pieces(int64_t rows, int32_t max_ctx, bool weights)
{
    if (max_ctx <= (rows >= 128 ? 2 * kAlone : kAlone)) return 1;
    int64_t n = std::max<int64_t>(1, kWave / rows);
    if (n * rows < kWave * 3 / 4 || max_ctx > n * 2048) n = (2 * kWave + rows - 1) / rows;
    n = std::max(n, std::min<int64_t>((max_ctx + 2047) / 2048, 4 * kWave / rows));
    n = std::min<int64_t>(n, std::max(16, max_ctx / 1024));
    if (!weights && n > kMostJoined && n <= 16 && max_ctx <= (rows >= 12 ? 4096 : 2048) && rows * kMostJoined <= kWave)
        n = kMostJoined;
    return n;
}

Plan4 plan4(const kvi_attention &a, int32_t R, int32_t max_ctx, bool weights)
{
    Plan4 pl{};
    const int G = a.q_heads / a.kv_heads;
    // two blocks of 8 heads share each decoded tile where registers allow
    pl.nt = G > 8 && a.head_dim <= 128 ? 2 : 1;
    pl.chunks = (G + 8 * pl.nt - 1) / (8 * pl.nt);
    const int64_t rows = (int64_t)R * a.kv_heads * pl.chunks;
    const int64_t want = pieces(rows, max_ctx, weights);
    int64_t span = (max_ctx + want - 1) / want;
    span = std::max<int64_t>(128, (span + 127) / 128 * 128);
    pl.span = (int)std::min<int64_t>(span, kLongest);
    pl.S = std::max(1, (int)(((int64_t)max_ctx + pl.span - 1) / pl.span));
    const size_t rq = (size_t)R * a.q_heads;
    // Up to 8 pieces of one wave are clusters, which join them: a launch less (us, 4
    // requests x 8 KV heads, 1024 keys 7.6 by a second kernel, 7.1; 24 x 2500 keys
    // 22.6, 21.0).  Not with weights, whose kernel joins on the side (24 x 1024 16.5,
    // 21.4), nor many clusters of 7, of which an odd number fits (8 x 2500 12.0, 13.0;
    // 4 x 1601 9.1, 8.3).
    pl.joined = !weights && pl.S > 1 && pl.S <= kMostJoined && rows * pl.S <= 4 * kPlanSms &&
                (pl.S != 7 || rows * 7 <= 2 * kPlanSms);
    pl.ml = pl.S > 1 && !pl.joined ? up256(rq * pl.S * a.head_dim * 4) : 0;
    pl.scores = pl.ml + up256(rq * pl.S * 8);
    pl.score_stride = (G + 1) & ~1;
    pl.total = pl.scores + (weights ? up256((size_t)R * a.kv_heads * max_ctx * pl.score_stride * 4) : 0);
    return pl;
}

// Workspace for these sizes and any smaller ones: fewer requests are cut into more
// pieces, so what a call needs does not go by its sizes, but with more than one
// piece a request there are 4 waves of blocks at most (`pieces`), and 16 pieces or
// one per 1024 keys.
size_t bytes4(const kvi_attention &a, int32_t R, int32_t max_ctx, bool weights)
{
    const Plan4 pl = plan4(a, R, max_ctx, weights);  // (its chunks and score rows go by the heads alone)
    int64_t parts = max_ctx > kLongest ? 2 * (int64_t)R : 0;
    if (max_ctx > kAlone)
        parts = std::max(parts, std::min(R * std::min<int64_t>(std::max(16, max_ctx / 1024), ((int64_t)max_ctx + 127) / 128),
                                         4 * kWave / ((int64_t)a.kv_heads * pl.chunks)));
    const size_t rows = (size_t)std::max<int64_t>(R, parts) * a.q_heads;
    return up256((size_t)parts * a.q_heads * a.head_dim * 4) + up256(rows * 8) +
           (weights ? up256((size_t)R * a.kv_heads * max_ctx * pl.score_stride * 4) : 0);
}

template <int NG, int NT, bool JOINED>
cudaError_t run4_as(const Decode4Params &p, int32_t R, cudaStream_t s)
{
    constexpr int bytes = Smem4<NG, NT>::kBytes;
    if (bytes > 48 * 1024) {
        const cudaError_t e = smem_opt_in(decode4_kernel<NG, NT, JOINED>, bytes);
        if (e != cudaSuccess) return e;
    }
    return launch_chained_clusters(decode4_kernel<NG, NT, JOINED>, JOINED ? p.S : 1,
                                   dim3((unsigned)p.S, (unsigned)(p.H * p.chunks), (unsigned)R), kWarps4 * 32, bytes, s, p);
}

template <int NG, int NT>
cudaError_t run4(const Decode4Params &p, int32_t R, cudaStream_t s)
{
    return p.joined ? run4_as<NG, NT, true>(p, R, s) : run4_as<NG, NT, false>(p, R, s);
}

cudaError_t launch_decode4(const Decode4Params &p, int nt, int32_t R, cudaStream_t s)
{
    switch (p.page.groups()) {
    case 1: return nt == 2 ? run4<1, 2>(p, R, s) : run4<1, 1>(p, R, s);
    case 2: return nt == 2 ? run4<2, 2>(p, R, s) : run4<2, 1>(p, R, s);
    case 3: return nt == 2 ? run4<3, 2>(p, R, s) : run4<3, 1>(p, R, s);
    case 4: return nt == 2 ? run4<4, 2>(p, R, s) : run4<4, 1>(p, R, s);
    case 5: return run4<5, 1>(p, R, s);
    case 6: return run4<6, 1>(p, R, s);
    case 7: return run4<7, 1>(p, R, s);
    default: return run4<8, 1>(p, R, s);
    }
}

bool sizes_ok(const kvi_attention *a, int32_t R, int32_t max_ctx)
{
    return a->head_dim % 32 == 0 && R >= 1 && R <= KVI_MAX_REQUESTS && max_ctx >= 0;
}

}  // namespace

}  // namespace kvi

using namespace kvi;

extern "C" size_t kvi_attn_decode4_workspace_bytes(const kvi_attention *a, int32_t R, int32_t max_ctx, int32_t weights)
{
    if (check_attention(a) != KVI_OK || !sizes_ok(a, R, max_ctx)) return 0;
    return bytes4(*a, R, max_ctx, weights != 0);
}

extern "C" kvi_status kvi_attn_decode4(const kvi_attention *a, int32_t R, const void *d_q, int64_t q_row_stride,
                                       const int32_t *d_ctx_lens, int32_t max_ctx, const int32_t *d_block_tables,
                                       int32_t max_blocks, const kvi_paged_cache *cache, int32_t layer, void *d_out,
                                       int64_t out_row_stride, float *d_weights, int64_t weights_stride, void *d_ws,
                                       size_t ws_bytes, int32_t *d_status, kvi_stream_t stream)
{
    kvi_status st = check_attention(a);
    if (st != KVI_OK) return st;
    st = cache4_check(a->kv_heads, a->head_dim, cache, layer);
    if (st != KVI_OK) return st;
    st = check_pages(cache, layer, R, max_blocks, d_block_tables);
    if (st != KVI_OK) return st;
    if (!sizes_ok(a, R, max_ctx)) return arg_error("max_ctx=%d must be >= 0", max_ctx);
    if (!d_q || unusable(d_ctx_lens, 4) || !d_out || unusable(d_status, 4) || (d_weights && unusable(d_weights, 4)))
        return arg_error("a required pointer (q, ctx_lens, out, status) is NULL, or one is misaligned");
    const int64_t wide = (int64_t)a->q_heads * a->head_dim;
    if (reinterpret_cast<uintptr_t>(d_q) % 16 || reinterpret_cast<uintptr_t>(d_out) % 16 || q_row_stride % 8 ||
        out_row_stride % 8 || q_row_stride < wide || out_row_stride < wide)
        return arg_error("q and out rows must be 16-byte aligned, with strides of at least q_heads * head_dim elements");
    if (d_weights && weights_stride < max_ctx)
        return arg_error("weights_stride=%lld is below max_ctx=%d", (long long)weights_stride, max_ctx);
    const Plan4 pl = plan4(*a, R, max_ctx, d_weights != nullptr);
    if ((int64_t)a->kv_heads * pl.chunks > 65535) return arg_error("kv_heads * head chunks is above 65535");
    if (!d_ws || ws_bytes < pl.total || reinterpret_cast<uintptr_t>(d_ws) % 256)
        return arg_error("workspace of %zu bytes (256-byte aligned) needed, %zu given", pl.total, ws_bytes);
    uint8_t *ws = static_cast<uint8_t *>(d_ws);
    Decode4Params p{};
    p.q = static_cast<const __nv_bfloat16 *>(d_q);
    p.q_stride = q_row_stride;
    p.ctx_lens = d_ctx_lens;
    p.max_ctx = max_ctx;
    p.max_blocks = max_blocks;
    p.block_tables = d_block_tables;
    p.num_blocks = cache->num_blocks;
    p.H = a->kv_heads;
    p.Hq = a->q_heads;
    p.G = a->q_heads / a->kv_heads;
    p.chunks = pl.chunks;
    p.page = Page4{cache->block_size, a->head_dim};
    p.pool = static_cast<const uint8_t *>(cache->layer_base[layer]);
    p.scale = a->scale * kLog2e;
    p.out = static_cast<__nv_bfloat16 *>(d_out);
    p.out_stride = out_row_stride;
    p.S = pl.S;
    p.span = pl.span;
    p.joined = pl.joined;
    p.po = reinterpret_cast<float *>(ws);
    p.ml = reinterpret_cast<float2 *>(ws + pl.ml);
    p.scores = d_weights ? reinterpret_cast<float *>(ws + pl.scores) : nullptr;
    p.score_stride = pl.score_stride;
    p.status = d_status;
    st = cuda_status(launch_decode4(p, pl.nt, R, stream), "kvi_attn_decode4");
    if (st != KVI_OK) return st;
    if ((pl.S == 1 || pl.joined) && (!d_weights || max_ctx == 0)) return st;
    WeightParams w{};
    JoinParams &j = w.join;
    j.po = p.po;
    j.ml = p.ml;
    j.S = pl.S;
    j.span = pl.span;
    j.R = R;
    j.q_heads = a->q_heads;
    j.D = a->head_dim;
    j.total_q = R;
    j.max_q = 1;
    j.ctx_lens = d_ctx_lens;
    j.max_ctx = max_ctx;
    j.max_blocks = max_blocks;
    j.block_size = cache->block_size;
    j.out = p.out;
    j.out_stride = out_row_stride;
    if (!d_weights) return cuda_status(launch_join(j, stream), "kvi_attn_decode4");
    w.join_blocks = pl.S > 1 && !pl.joined ? (a->q_heads + kJoinWarps - 1) / kJoinWarps : 0;
    w.key_blocks = (max_ctx + kKeysBlock - 1) / kKeysBlock;
    w.scores = p.scores;
    w.score_stride = pl.score_stride;
    w.H = p.H;
    w.G = p.G;
    w.w = d_weights;
    w.stride = weights_stride;
    const dim3 grid((unsigned)(w.join_blocks + (int64_t)w.key_blocks * w.H), (unsigned)R);
    return cuda_status(launch_chained(finish_kernel, grid, kJoinWarps * 32, 0, stream, w), "kvi_attn_decode4");
}
