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
// this instruction's fragment order, so a lane loads its share of 16 tokens
// with a few wide loads straight into registers.
//   K: a group's product is taken of the bare codes and then scaled by the
//      key's step in float32 (step * code has 12 significant bits and would
//      not fit a bf16 operand).
//   V: the step belongs to (key, group), and a key is summed over, so P is
//      scaled: P and P * step round to bf16, as any P on tensor cores does.
//   A code c in the low nibble of a 16-bit half, or'ed with 0x4300, is the
//      bf16 number 128 + c; 136 is subtracted exactly.
// A warp takes tiles of 16 keys in turn with a softmax of its own; the warps of
// a block join at the end, and blocks that share a request's keys join in a
// second kernel.
#include <cuda_runtime.h>

#include <algorithm>

#include "kvi_attn.cuh"

namespace kvi {

namespace {

constexpr int kWarps4 = 4;
constexpr int kPlanSms = 152;

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
    float *po;
    float2 *ml;
    float *scores;   // [R][H][max_ctx][score_stride] or null
    int32_t score_stride;
    int32_t *status;
};

// N 32-bit words from p, with the widest loads their count allows (p is
// aligned to that width).
template <int N>
__device__ __forceinline__ void load_words(uint32_t (&w)[N], const uint8_t *p)
{
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p) + i);
            w[4 * i] = v.x;
            w[4 * i + 1] = v.y;
            w[4 * i + 2] = v.z;
            w[4 * i + 3] = v.w;
        }
    } else if constexpr (N % 2 == 0) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p) + i);
            w[2 * i] = v.x;
            w[2 * i + 1] = v.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = __ldg(reinterpret_cast<const uint32_t *>(p) + i);
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
            w[i] = (uint32_t)__ldg(h + 2 * i) | (2 * i + 1 < N ? (uint32_t)__ldg(h + 2 * i + 1) << 16 : 0u);
    }
}

// The codes in nibbles 0 and 4 of w as two bf16 numbers
__device__ __forceinline__ uint32_t codes_bf16x2(uint32_t w)
{
    const uint32_t b = (w & 0x000f000fu) | 0x43004300u;
    const uint32_t off = 0x43084308u;  // 136, 136
    const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&b),
                                     *reinterpret_cast<const __nv_bfloat162 *>(&off));
    return *reinterpret_cast<const uint32_t *>(&v);
}

// This lane's share of 16 tokens of a page.
template <int NG>
struct Tile4 {
    uint32_t kc[2][NG];            // keys lane / 4 and + 8
    uint32_t ks[2][(NG + 1) / 2];  // their steps
    uint32_t vc[2][NG];            // token pairs lane % 4 and + 4
    uint32_t vs[2][NG];            // their steps (both tokens of the pair)
    bool live;                     // false: nothing was read (bad block)
};

template <int NG>
__device__ __forceinline__ void load_tile(Tile4<NG> &x, const Decode4Params &p, const int32_t *table, int h, int tile)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int k0 = tile * 16;
    const int b = table[k0 / p.page.B];
    x.live = b >= 0 && b < p.num_blocks;
    if (!x.live) {
        if (lane == 0) record_status(p.status, KVI_ERR_OUT_OF_RANGE);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int j = 0; j < NG; ++j) x.kc[i][j] = x.vc[i][j] = x.vs[i][j] = 0;
#pragma unroll
            for (int j = 0; j < (NG + 1) / 2; ++j) x.ks[i][j] = 0;
        }
        return;
    }
    const uint8_t *page = p.pool + ((int64_t)b * p.H + h) * p.page.bytes();
    const int off = k0 % p.page.B;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int key = off + g + 8 * i, pair = off / 2 + t + 4 * i;
        load_words<NG>(x.kc[i], page + (int64_t)key * (NG * 16) + t * (NG * 4));
        load_words<NG>(x.vc[i], page + p.page.v_codes() + (int64_t)pair * (NG * 32) + g * (NG * 4));
        load_halves<NG>(x.ks[i], page + p.page.k_steps() + (int64_t)key * (NG * 2));
        load_words<NG>(x.vs[i], page + p.page.v_steps() + (int64_t)pair * (NG * 4));
    }
}

template <int NG, int NT>
__global__ void __launch_bounds__(kWarps4 * 32) decode4_kernel(const __grid_constant__ Decode4Params p)
{
    constexpr int D = NG * 32;
    __shared__ float s_o[kWarps4][8 * NT][D + 4];
    __shared__ float s_m[kWarps4][8 * NT], s_l[kWarps4][8 * NT];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int split = blockIdx.x;
    const int h = blockIdx.y / p.chunks, c0 = (blockIdx.y % p.chunks) * 8 * NT;  // first head of the group
    const int r = blockIdx.z;
    RequestSpan rq;
    if (!request_span(r, nullptr, (int)gridDim.z, 1, p.ctx_lens, p.max_ctx, p.max_blocks, p.page.B, rq)) {
        if (tid == 0) record_status(p.status, KVI_ERR_OUT_OF_RANGE);
        return;
    }
    const int from = split * p.span, to = min(rq.ctx, from + p.span);
    if (from >= to && split > 0) return;  // split 0 writes the zeros of an empty cache
    const bool whole = rq.ctx <= p.span;

    // Q as B fragments: word (a, b) of group j is channels 32 j + 8 t + 2 a + b
    // and + 4, the order of the codes' nibbles
    uint32_t qf[NT][2 * NG][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int head = c0 + 8 * nt + g;
        const __nv_bfloat16 *q = p.q + (int64_t)r * p.q_stride + ((int64_t)h * p.G + head) * D + 8 * t;
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (head < p.G) v = __ldg(reinterpret_cast<const uint4 *>(q + 32 * j));
            // v = channels (0,1) (2,3) (4,5) (6,7)
            qf[nt][2 * j][0] = __byte_perm(v.x, v.z, 0x5410);      // 0, 4
            qf[nt][2 * j][1] = __byte_perm(v.x, v.z, 0x7632);      // 1, 5
            qf[nt][2 * j + 1][0] = __byte_perm(v.y, v.w, 0x5410);  // 2, 6
            qf[nt][2 * j + 1][1] = __byte_perm(v.y, v.w, 0x7632);  // 3, 7
        }
    }
    float o[NT][2 * NG][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < 2 * NG; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[nt][i][j] = 0.f;
        m[nt][0] = m[nt][1] = neg_inf();
        l[nt][0] = l[nt][1] = 0.f;
    }

    const int32_t *table = p.block_tables + (int64_t)r * p.max_blocks;
    const int t1 = (to + 15) / 16;
    int tile = from / 16 + warp;
    Tile4<NG> x;
    if (tile < t1) load_tile<NG>(x, p, table, h, tile);
    for (; tile < t1; tile += kWarps4) {
        Tile4<NG> y;
        if (tile + kWarps4 < t1) load_tile<NG>(y, p, table, h, tile + kWarps4);
        // ---- scores: rows g and g + 8 of the tile, heads 2 t and 2 t + 1
        float s[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[nt][i] = 0.f;
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            const float k0 = (j & 1) ? bf16_hi(x.ks[0][j / 2]) : bf16_lo(x.ks[0][j / 2]);
            const float k1 = (j & 1) ? bf16_hi(x.ks[1][j / 2]) : bf16_lo(x.ks[1][j / 2]);
            float part[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) part[nt][i] = 0.f;
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                const uint32_t a0 = codes_bf16x2(x.kc[0][j] >> (8 * a)), a1 = codes_bf16x2(x.kc[1][j] >> (8 * a));
                const uint32_t a2 = codes_bf16x2(x.kc[0][j] >> (8 * a + 4)), a3 = codes_bf16x2(x.kc[1][j] >> (8 * a + 4));
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma16816(part[nt], a0, a1, a2, a3, qf[nt][2 * j + a][0], qf[nt][2 * j + a][1]);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                s[nt][0] = fmaf(k0, part[nt][0], s[nt][0]);
                s[nt][1] = fmaf(k0, part[nt][1], s[nt][1]);
                s[nt][2] = fmaf(k1, part[nt][2], s[nt][2]);
                s[nt][3] = fmaf(k1, part[nt][3], s[nt][3]);
            }
        }
        const int key = tile * 16 + g;
        const bool in0 = x.live && key < to, in1 = x.live && key + 8 < to;
        bool move = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < 4; ++i) s[nt][i] = (i < 2 ? in0 : in1) ? s[nt][i] * p.scale : neg_inf();
            move |= fmaxf(s[nt][0], s[nt][2]) > m[nt][0] + kLazy || fmaxf(s[nt][1], s[nt][3]) > m[nt][1] + kLazy;
        }
        if (p.scores) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int head = c0 + 8 * nt + 2 * t;
                float *sc = p.scores + (((int64_t)r * p.H + h) * p.max_ctx + key) * p.score_stride + head;
                if (head < p.score_stride) {
                    if (key < to) *reinterpret_cast<float2 *>(sc) = make_float2(s[nt][0], s[nt][1]);
                    if (key + 8 < to)
                        *reinterpret_cast<float2 *>(sc + 8 * p.score_stride) = make_float2(s[nt][2], s[nt][3]);
                }
            }
        }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float top = fmaxf(s[nt][c], s[nt][c + 2]);
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                    // each column goes by its own scores alone
                    if (!(top > m[nt][c] + kLazy)) continue;
                    const float f = exp2_fast(m[nt][c] - top);
                    m[nt][c] = top;
                    l[nt][c] *= f;
#pragma unroll
                    for (int i = 0; i < 2 * NG; ++i) {
                        o[nt][i][c] *= f;
                        o[nt][i][c + 2] *= f;
                    }
                }
        }
        // ---- weights, as B fragments: keys 2 t, 2 t + 1 (and + 8) of head g
        uint32_t b0[NT], b1[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float m0 = m[nt][0] == neg_inf() ? 0.f : m[nt][0], m1 = m[nt][1] == neg_inf() ? 0.f : m[nt][1];
            const float p0 = exp2_fast(s[nt][0] - m0), p1 = exp2_fast(s[nt][1] - m1);
            const float p2 = exp2_fast(s[nt][2] - m0), p3 = exp2_fast(s[nt][3] - m1);
            l[nt][0] += p0 + p2;
            l[nt][1] += p1 + p3;
            b0[nt] = transpose8x8(pack_bf16(p0, p1));
            b1[nt] = transpose8x8(pack_bf16(p2, p3));
        }
        // slots past the end have weight 0, but their steps may hold anything
        if (tile * 16 + 16 > to) {
            const uint32_t lo = tile * 16 + 2 * t < to ? 0x0000ffffu : 0u, hi = tile * 16 + 2 * t + 1 < to ? 0xffff0000u : 0u;
            const uint32_t lo8 = tile * 16 + 2 * t + 8 < to ? 0x0000ffffu : 0u;
            const uint32_t hi8 = tile * 16 + 2 * t + 9 < to ? 0xffff0000u : 0u;
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                x.vs[0][j] &= lo | hi;
                x.vs[1][j] &= lo8 | hi8;
            }
        }
        // ---- output: channels 32 j + 4 g + 2 a (+ 1), heads 2 t and 2 t + 1
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            uint32_t w0[NT], w1[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                w0[nt] = mul_bf16x2(b0[nt], x.vs[0][j]);
                w1[nt] = mul_bf16x2(b1[nt], x.vs[1][j]);
            }
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                const uint32_t a0 = codes_bf16x2(x.vc[0][j] >> (8 * a)), a1 = codes_bf16x2(x.vc[0][j] >> (8 * a + 4));
                const uint32_t a2 = codes_bf16x2(x.vc[1][j] >> (8 * a)), a3 = codes_bf16x2(x.vc[1][j] >> (8 * a + 4));
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma16816(o[nt][2 * j + a], a0, a1, a2, a3, w0[nt], w1[nt]);
            }
        }
        x = y;
    }

    // ---- the block's warps join
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], off);
            const int n = 8 * nt + 2 * t + c;
            if (g == 0) {
                s_m[warp][n] = m[nt][c];
                s_l[warp][n] = l[nt][c];
            }
#pragma unroll
            for (int j = 0; j < NG; ++j)
                *reinterpret_cast<float4 *>(&s_o[warp][n][32 * j + 4 * g]) =
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
            acc.x += s_o[w][n][d] * f;
            acc.y += s_o[w][n][d + 1] * f;
        }
        const int64_t row = (int64_t)r * p.Hq + (int64_t)h * p.G + c0 + n;
        if (whole) {
            const float inv = L == 0.f ? 0.f : 1.f / L;
            *reinterpret_cast<uint32_t *>(p.out + (int64_t)r * p.out_stride + ((int64_t)h * p.G + c0 + n) * D + d) =
                pack_bf16(acc.x * inv, acc.y * inv);
        } else {
            *reinterpret_cast<float2 *>(p.po + (row * p.S + split) * D + d) = acc;
        }
        if (d == 0 && (!whole || p.scores)) p.ml[row * p.S + split] = make_float2(M, L);
    }
}

// ------------------------------------------------------ accumulated weights

struct WeightParams {
    const float *scores;
    int32_t score_stride;
    const float2 *ml;
    int32_t S, span;
    int32_t H, Hq, G;
    const int32_t *ctx_lens;
    int32_t max_ctx, max_blocks, block_size;
    float *w;
    int64_t stride;
};

constexpr int kWeightThreads = 256;

// weights[r][h][p] += sum over the group's heads of 2^(s_p - M) / L
__global__ void __launch_bounds__(kWeightThreads) weight_kernel(const WeightParams p)
{
    __shared__ float s_ref[KVI_MAX_ATTN_GROUP], s_inv[KVI_MAX_ATTN_GROUP];
    pdl_wait();
    const int h = blockIdx.y, r = blockIdx.z, tid = threadIdx.x;
    RequestSpan rq;
    if (!request_span(r, nullptr, (int)gridDim.z, 1, p.ctx_lens, p.max_ctx, p.max_blocks, p.block_size, rq)) return;
    if ((int64_t)blockIdx.x * kWeightThreads >= rq.ctx) return;
    const int pieces = (rq.ctx + p.span - 1) / p.span;
    for (int g = tid; g < p.G; g += kWeightThreads) {
        const float2 *ml = p.ml + ((int64_t)r * p.Hq + (int64_t)h * p.G + g) * p.S;
        float M = neg_inf();
        for (int s = 0; s < pieces; ++s) M = fmaxf(M, ml[s].x);
        const float ref = M == neg_inf() ? 0.f : M;
        float L = 0.f;
        for (int s = 0; s < pieces; ++s) L += ml[s].y * exp2_fast(ml[s].x - ref);
        s_ref[g] = ref;
        s_inv[g] = L == 0.f ? 0.f : 1.f / L;
    }
    __syncthreads();
    const int key = blockIdx.x * kWeightThreads + tid;
    if (key >= rq.ctx) return;
    const float *s = p.scores + (((int64_t)r * p.H + h) * p.max_ctx + key) * p.score_stride;
    float sum = 0.f;
    for (int g = 0; g < p.G; ++g) sum += exp2_fast(s[g] - s_ref[g]) * s_inv[g];
    float *w = p.w + ((int64_t)r * p.H + h) * p.stride + key;
    *w += sum;
}

// -------------------------------------------------------------------- host

struct Plan4 {
    int nt, chunks, S, span;
    size_t ml, scores, total;  // byte offsets after the partial outputs
    int score_stride;
};

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

Plan4 plan4(const kvi_attention &a, int32_t R, int32_t max_ctx, bool weights)
{
    Plan4 pl{};
    const int G = a.q_heads / a.kv_heads;
    // two blocks of 8 heads share each decoded tile where registers allow
    pl.nt = G > 8 && a.head_dim <= 128 ? 2 : 1;
    pl.chunks = (G + 8 * pl.nt - 1) / (8 * pl.nt);
    // enough blocks for four on every SM, but none below 256 keys (four tiles a warp)
    const int64_t rows = (int64_t)R * a.kv_heads * pl.chunks;
    const int64_t want = std::max<int64_t>(1, (8 * kPlanSms + rows - 1) / rows);
    int64_t span = (max_ctx + want - 1) / want;
    span = std::max<int64_t>(256, (span + 63) / 64 * 64);
    pl.span = (int)std::min<int64_t>(span, 1 << 30);
    pl.S = std::max(1, (int)(((int64_t)max_ctx + pl.span - 1) / pl.span));
    const size_t rq = (size_t)R * a.q_heads;
    pl.ml = pl.S > 1 ? up256(rq * pl.S * a.head_dim * 4) : 0;
    pl.scores = pl.ml + up256(rq * pl.S * 8);
    pl.score_stride = (G + 1) & ~1;
    pl.total = pl.scores + (weights ? up256((size_t)R * a.kv_heads * max_ctx * pl.score_stride * 4) : 0);
    return pl;
}

template <int NG, int NT>
cudaError_t run4(const Decode4Params &p, int32_t R, cudaStream_t s)
{
    decode4_kernel<NG, NT><<<dim3((unsigned)p.S, (unsigned)(p.H * p.chunks), (unsigned)R), kWarps4 * 32, 0, s>>>(p);
    return cudaGetLastError();
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
    return plan4(*a, R, max_ctx, weights != 0).total;
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
    p.po = reinterpret_cast<float *>(ws);
    p.ml = reinterpret_cast<float2 *>(ws + pl.ml);
    p.scores = d_weights ? reinterpret_cast<float *>(ws + pl.scores) : nullptr;
    p.score_stride = pl.score_stride;
    p.status = d_status;
    st = cuda_status(launch_decode4(p, pl.nt, R, stream), "kvi_attn_decode4");
    if (st != KVI_OK) return st;
    if (pl.S > 1) {
        JoinParams j{};
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
        st = cuda_status(launch_join(j, stream), "kvi_attn_decode4");
        if (st != KVI_OK) return st;
    }
    if (d_weights && max_ctx > 0) {
        WeightParams w{};
        w.scores = p.scores;
        w.score_stride = pl.score_stride;
        w.ml = p.ml;
        w.S = pl.S;
        w.span = pl.span;
        w.H = p.H;
        w.Hq = p.Hq;
        w.G = p.G;
        w.ctx_lens = d_ctx_lens;
        w.max_ctx = max_ctx;
        w.max_blocks = max_blocks;
        w.block_size = cache->block_size;
        w.w = d_weights;
        w.stride = weights_stride;
        weight_kernel<<<dim3((unsigned)((max_ctx + kWeightThreads - 1) / kWeightThreads), (unsigned)p.H, (unsigned)R),
                        kWeightThreads, 0, stream>>>(w);
        st = cuda_status(cudaGetLastError(), "kvi_attn_decode4");
    }
    return st;
}
