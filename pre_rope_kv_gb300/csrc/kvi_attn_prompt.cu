// kvi_attn_prompt.cu -- causal attention of packed prompts over the paged
// bf16 cache: row i of a request's n rows sees the positions <= ctx - n + i.
//
// A KV head's query rows are its group's heads for every token, token first:
// row = token * G + head, so the rows that read the same keys share a tile.
//
// Long prompts run on the tensor cores' tiles (kvi_attn_tile.cu).  rows_kernel
// here takes 8 or 16 rows a block, for few rows and for the page and head sizes
// that the tiles do not take.  Its products are S^T = K Q^T (16 keys x 8 rows) and
// O^T = V^T P^T, as with few rows it is K and V that fill the matrix instruction's
// M.  Each warp streams its own tiles of 16 keys (16-byte asynchronous copies into
// a ring of its own, so no block-wide wait) and keeps a softmax of its own; the
// block's warps join at the end, and blocks that share a request's keys through one
// another's shared memory as a cluster, or in a second kernel.  Where a block's rows are all there are (decoding steps) the
// cache's bytes bound it: 64 requests x 1.5 k keys, 8 KV heads of 128 channels,
// 71 us, 5.3 TB/s.
#include <cuda_runtime.h>

#include <algorithm>

#include "kvi_attn.cuh"

namespace kvi {

namespace {

constexpr int kRowWarps = 4;
constexpr int kRowStages = 2;  // (three blocks fit an SM; with 3: two blocks, 64 x 1.5 k keys 78 us instead of 71)

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

// 16 bytes to shared memory, or zeros when `bytes` is 0
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}

__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t a)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}

__device__ __forceinline__ uint32_t not_finite(uint32_t w)  // bits 15 / 31: that half is an infinity or NaN
{
    const uint32_t e = w & 0x7f807f80u;
    return ((e + 0x00800080u) & 0x80008000u);
}

// Shared memory of a block: the warps' rings (rows padded by 16 bytes, so that
// the 8 rows of a matrix load fall into different banks), reused for the join.
template <int DP, int NT>
struct RowsSmem {
    static constexpr int kPitch = DP * 2 + 16;
    static constexpr int kStage = 2 * 16 * kPitch;  // K then V of 16 keys
    static constexpr int kRing = kRowStages * kStage;
    static constexpr int kSum = kRowWarps * 8 * NT * (DP + 4) * 4;  // then the block's own
    static constexpr int kJoin = kSum + 8 * NT * DP * 4;
    static constexpr int kBytes = kRowWarps * kRing > kJoin ? kRowWarps * kRing : kJoin;
};

// DP: the head size rounded up to 32, 64, 128 or 256 (the rest reads as zero);
// 8 * NT rows per block.  JOINED: a chunk's pieces are a cluster, which joins them.
template <int DP, int NT, bool JOINED>
__global__ void __launch_bounds__(kRowWarps * 32) rows_kernel(const __grid_constant__ PromptParams p)
{
    using Sm = RowsSmem<DP, NT>;
    constexpr int KS = DP / 16, CH = DP / 8;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ uint32_t s_here[kRowWarps][kRowStages];
    __shared__ float s_m[kRowWarps][8 * NT], s_l[kRowWarps][8 * NT];
    __shared__ float2 s_ml[8 * NT];  // of the block
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int split = blockIdx.x % p.S, chunk = (blockIdx.x / p.S) % p.chunks, h = blockIdx.x / p.S / p.chunks;
    const int r = blockIdx.y;
    pdl_wait();
    pdl_launch_dependents();
    RequestSpan rq;
    if (!request_span(r, p.q_start, p.total_q, p.max_q, p.ctx_lens, p.max_ctx, p.max_blocks, p.B, rq)) {
        if (tid == 0) record_status(p.status, KVI_ERR_OUT_OF_RANGE);
        return;
    }
    const int rows = rq.n_q * p.G, row0 = chunk * 8 * NT;
    if (row0 >= rows) return;
    const int pieces = max(1, (rq.ctx + p.span - 1) / p.span);
    if (split >= pieces) {
        if (JOINED && pieces > 1) {  // (the others of the cluster count on it)
            cluster_sync();
            cluster_sync();
        }
        return;
    }
    const int seen_by_0 = rq.ctx - rq.n_q;  // last position that token 0 sees
    const int end = min(rq.ctx, seen_by_0 + (min(rows, row0 + 8 * NT) - 1) / p.G + 1);
    const int from = split * p.span, to = min(end, from + p.span);
    const bool whole = pieces == 1;

    // the rows' last visible positions: columns 2 t, 2 t + 1 of each n-tile
    int last[NT][2];
    int least = INT32_MAX;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int row = row0 + 8 * nt + 2 * t + c;
            last[nt][c] = row < rows ? seen_by_0 + row / p.G : -1;
            if (row < rows) least = min(least, last[nt][c]);
        }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) least = min(least, __shfl_xor_sync(0xffffffffu, least, o));

    uint32_t qf[NT][KS][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int row = row0 + 8 * nt + g;
        const bool in = row < rows;
        const __nv_bfloat16 *q =
            p.q + (int64_t)(rq.q0 + (in ? row / p.G : 0)) * p.q_stride + ((int64_t)h * p.G + row % p.G) * p.D + 2 * t;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            const bool real = in && 16 * k < p.D;  // D is a multiple of 16
            qf[nt][k][0] = real ? *reinterpret_cast<const uint32_t *>(q + 16 * k) : 0u;
            qf[nt][k][1] = real ? *reinterpret_cast<const uint32_t *>(q + 16 * k + 8) : 0u;
        }
    }
    float o[NT][KS][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[nt][i][j] = 0.f;
        m[nt][0] = m[nt][1] = neg_inf();
        l[nt][0] = l[nt][1] = 0.f;
    }

    // ---- this warp's tiles: from / 16 + warp, + kRowWarps, ...
    uint8_t *ring = smem + warp * Sm::kRing;
    if (p.D < DP) {  // channels past D: copied never, zero for good
        for (int i = lane; i < kRowStages * 32; i += 32)
            for (int c = p.D / 8; c < CH; ++c)
                *reinterpret_cast<uint4 *>(ring + i * Sm::kPitch + c * 16) = make_uint4(0, 0, 0, 0);
    }
    const int32_t *table = p.block_tables + (int64_t)r * p.max_blocks;
    const int64_t plane = (int64_t)p.num_blocks * p.B * p.H * p.D;
    const int t0 = from / 16 + warp, t1 = (to + 15) / 16;
    const uint32_t ring_a = smem_addr(ring);

    // block of key `lane` (mod 16) of a tile; -1 outside
    auto block_of = [&](int tile) {
        const int key = tile * 16 + (lane & 15);
        return tile < t1 && key < rq.ctx ? table[key / p.B] : -1;
    };
    auto issue = [&](int tile, int stage, int block) {
        const int key = tile * 16 + (lane & 15);
        const bool asked = tile < t1 && key < rq.ctx;
        const bool here = asked && block >= 0 && block < p.num_blocks;
        if (asked && !here) record_status(p.status, KVI_ERR_OUT_OF_RANGE);
        const int64_t at = here ? (((int64_t)block * p.B + key % p.B) * p.H + h) * p.D : -1;
        const uint32_t mask = __ballot_sync(0xffffffffu, here);
        if (lane == 0) s_here[warp][stage] = mask & 0xffffu;
        if (tile < t1) {
#pragma unroll 4
            for (int i = 0; i < 16 * CH / 32; ++i) {
                const int c = i * 32 + lane, row = c / CH, col = c % CH;
                const int64_t a = __shfl_sync(0xffffffffu, at, row);
                if (col * 8 < p.D) {
                    const __nv_bfloat16 *src = p.pool + (a < 0 ? 0 : a + col * 8);
                    const uint32_t dst = ring_a + stage * Sm::kStage + row * Sm::kPitch + col * 16;
                    copy16(dst, src, a < 0 ? 0 : 16);
                    copy16(dst + 16 * Sm::kPitch, src + (a < 0 ? 0 : plane), a < 0 ? 0 : 16);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int s = 0; s < kRowStages - 1; ++s) issue(t0 + s * kRowWarps, s, block_of(t0 + s * kRowWarps));
    int next_block = block_of(t0 + (kRowStages - 1) * kRowWarps);
    int stage = 0;
    for (int tile = t0; tile < t1; tile += kRowWarps) {
        const int ahead = tile + (kRowStages - 1) * kRowWarps;
        issue(ahead, stage == 0 ? kRowStages - 1 : stage - 1, next_block);
        next_block = block_of(ahead + kRowWarps);
        asm volatile("cp.async.wait_group %0;" ::"n"(kRowStages - 1) : "memory");
        __syncwarp();
        const uint32_t ka = ring_a + stage * Sm::kStage, va = ka + 16 * Sm::kPitch;
        // ---- scores: keys g and g + 8, rows 2 t and 2 t + 1 of each n-tile
        float s[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[nt][i] = 0.f;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            uint32_t a[4];
            ldsm4(a, ka + (lane & 15) * Sm::kPitch + (2 * k + (lane >> 4)) * 16);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816(s[nt], a[0], a[1], a[2], a[3], qf[nt][k][0], qf[nt][k][1]);
        }
        const int key = tile * 16 + g;
        const uint32_t here = s_here[warp][stage];
        bool move = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int kk = key + (i >> 1) * 8;
                const bool see = kk <= last[nt][i & 1] && ((here >> (g + (i >> 1) * 8)) & 1u);
                s[nt][i] = see ? s[nt][i] * p.scale : neg_inf();
            }
            move |= fmaxf(s[nt][0], s[nt][2]) > m[nt][0] + kLazy || fmaxf(s[nt][1], s[nt][3]) > m[nt][1] + kLazy;
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
                    for (int i = 0; i < KS; ++i) {
                        o[nt][i][c] *= f;
                        o[nt][i][c + 2] *= f;
                    }
                }
            __syncwarp();  // the next matrix instruction wants the warp as one
        }
        // ---- P rounds to bf16 for the second product, whose operands are of one type
        // and V's is bf16: each weight by up to 2^-8 of itself, which leaves the output
        // 0.0023 off (mean square, of it) where its own rounding alone leaves 0.0017.  The
        // sum takes P unrounded.
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
        // a tile that some row sees only in part: an infinity or NaN among its
        // values must not reach the rows that do not see it (0 * inf)
        const bool partly = tile * 16 + 15 > least;
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            uint32_t a[4];
            ldsm4_t(a, va + ((lane & 7) + (lane >> 4) * 8) * Sm::kPitch + (2 * i + ((lane >> 3) & 1)) * 16);
            if (partly) {
                uint32_t bad = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t f = not_finite(a[j]);
                    bad |= f;
                    a[j] &= ~((f >> 15) * 0xffffu);
                }
                if (__any_sync(0xffffffffu, bad != 0)) {
                    for (int kk = 0; kk < 16; ++kk)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {  // channels 16 i + g and + 8
                            const uint16_t *v = reinterpret_cast<const uint16_t *>(
                                ring + stage * Sm::kStage + (16 + kk) * Sm::kPitch + (16 * i + g + 8 * j) * 2);
                            if ((*v & 0x7f80u) != 0x7f80u) continue;
                            const float x = __uint_as_float((uint32_t)*v << 16);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int c = 0; c < 2; ++c)
                                    if (tile * 16 + kk <= last[nt][c]) o[nt][i][2 * j + c] += x;
                        }
                    __syncwarp();
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816(o[nt][i], a[0], a[1], a[2], a[3], b0[nt], b1[nt]);
        }
        __syncwarp();  // the stage has been read
        stage = stage + 1 == kRowStages ? 0 : stage + 1;
    }

    // ---- the block's warps join, in the rings' memory
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    float *s_o = reinterpret_cast<float *>(smem);
    constexpr int kO = DP + 4;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], off);
            const int n = 8 * nt + 2 * t + c;
            if (g == 0) {
                s_m[warp][n] = m[nt][c];
                s_l[warp][n] = l[nt][c];
            }
            float *dst = s_o + (warp * 8 * NT + n) * kO + g;
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                dst[16 * i] = o[nt][i][c];
                dst[16 * i + 8] = o[nt][i][c + 2];
            }
        }
    __syncthreads();
    const int half = p.D / 2;
    for (int i = tid; i < 8 * NT * half; i += kRowWarps * 32) {
        const int n = i / half, d = (i % half) * 2, row = row0 + n;
        if (row >= rows) break;
        float M = neg_inf();
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) M = fmaxf(M, s_m[w][n]);
        const float ref = M == neg_inf() ? 0.f : M;
        float L = 0.f;
        float2 acc = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) {
            const float f = exp2_fast(s_m[w][n] - ref);
            const float *src = s_o + (w * 8 * NT + n) * kO + d;
            L += s_l[w][n] * f;
            acc.x += src[0] * f;
            acc.y += src[1] * f;
        }
        const int64_t token = rq.q0 + row / p.G;
        const int head = h * p.G + row % p.G;
        const int64_t at = token * p.Hq + head;
        if (whole) {
            const float inv = L == 0.f ? 0.f : 1.f / L;
            *reinterpret_cast<uint32_t *>(p.out + token * p.out_stride + (int64_t)head * p.D + d) =
                pack_bf16(acc.x * inv, acc.y * inv);
            if (p.lse && d == 0) p.lse[at] = L == 0.f ? neg_inf() : (M + log2f(L)) * kLn2;
        } else if (JOINED) {
            *reinterpret_cast<float2 *>(smem + Sm::kSum + (n * DP + d) * 4) = acc;
            if (d == 0) s_ml[n] = make_float2(M, L);
        } else {
            const int64_t part = ((p.by_request ? (int64_t)r * p.max_q : rq.q0) + row / p.G) * p.Hq + head;
            *reinterpret_cast<float2 *>(p.po + (part * p.S + split) * p.D + d) = acc;
            if (d == 0) p.ml[part * p.S + split] = make_float2(M, L);
        }
    }
    if (!JOINED || whole) return;
    // ---- each block of the cluster that has keys joins a part of the channels
    cluster_sync();
    for (int i = split * kRowWarps * 32 + tid; i < 8 * NT * half; i += pieces * kRowWarps * 32) {
        const int n = i / half, d = (i % half) * 2, row = row0 + n;
        if (row >= rows) break;
        float2 ml[kMostJoined], part[kMostJoined];
        float M = neg_inf();
#pragma unroll
        for (int k = 0; k < kMostJoined; ++k) {
            if (k >= pieces) continue;
            ml[k] = load_of_block(smem_addr(&s_ml[n]), k);
            part[k] = load_of_block(smem_addr(smem + Sm::kSum + (n * DP + d) * 4), k);
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
        const int64_t token = rq.q0 + row / p.G;
        const int head = h * p.G + row % p.G;
        const float inv = L == 0.f ? 0.f : 1.f / L;
        *reinterpret_cast<uint32_t *>(p.out + token * p.out_stride + (int64_t)head * p.D + d) =
            pack_bf16(acc.x * inv, acc.y * inv);
        if (p.lse && d == 0) p.lse[token * p.Hq + head] = L == 0.f ? neg_inf() : (M + log2f(L)) * kLn2;
    }
    cluster_sync();  // no block leaves while its sums are read
}

// -------------------------------------------------------------------- host

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

struct PromptPlan {
    bool tiles;  // the form of kvi_attn_tile.cu
    int dp, nt;
    int64_t chunks;
    int S, span;
    bool joined;
    size_t ml, total;
};

constexpr int kLongest = 1 << 30;              // keys of a piece at most
constexpr int kRowsWanted = 4 * kPlanSms;      // blocks of the rows form
constexpr int kRowsAlone = 256, kTilesAlone = 384;

// Rows whose partial results are kept: of q, but no more than the requests have
int64_t part_rows(int32_t R, int32_t total_q, int32_t max_q) { return std::min<int64_t>(total_q, (int64_t)R * max_q); }

// `splits` pieces of the keys are wanted, none below `least` keys, and none at
// all up to `alone` keys, which cost no more than the join does (2 us).
void plan_split(PromptPlan &pl, const kvi_attention &a, int64_t rows, int32_t max_ctx, int64_t splits, int alone, int least)
{
    if (max_ctx <= alone) splits = 1;
    int64_t span = (max_ctx + splits - 1) / splits;
    span = std::max<int64_t>(least, (span + 127) / 128 * 128);
    pl.span = (int)std::min<int64_t>(span, kLongest);
    pl.S = std::max(1, (int)(((int64_t)max_ctx + pl.span - 1) / pl.span));
    if (pl.S > 1) {
        const size_t n_rows = (size_t)rows * a.q_heads;
        pl.ml = up256(n_rows * pl.S * a.head_dim * 4);
        pl.total = pl.ml + up256(n_rows * pl.S * 8);
    }
}

PromptPlan plan_rows(const kvi_attention &a, int32_t R, int32_t total_q, int32_t max_q, int32_t max_ctx)
{
    PromptPlan pl{};
    const int G = a.q_heads / a.kv_heads;
    pl.dp = a.head_dim <= 32 ? 32 : a.head_dim <= 64 ? 64 : a.head_dim <= 128 ? 128 : 256;
    const int64_t rows = (int64_t)max_q * G;
    pl.nt = rows > 8 && pl.dp <= 128 ? 2 : 1;
    pl.chunks = std::max<int64_t>(1, (rows + 8 * pl.nt - 1) / (8 * pl.nt));
    // blocks for four on every SM; short ones only where there are few (16 requests
    // of one token, 512 keys: 14 us in pieces of 128, 12 us in pieces of 256)
    const int64_t n = (int64_t)R * a.kv_heads * pl.chunks;
    plan_split(pl, a, part_rows(R, total_q, max_q), max_ctx, std::max<int64_t>(1, (kRowsWanted + n - 1) / n), kRowsAlone,
               2 * n > kPlanSms ? 256 : 128);
    // Up to 8 pieces are clusters, which join them, while these find room at once
    // (three blocks an SM; us, one token, 8 KV heads of 128 channels, by a second
    // kernel and so: 1 request x 1024 keys 7.5, 6.7; 8 x 700, 384 blocks, 10.0, 8.9;
    // 8 x 1601, 448 blocks, 12.8, 19.5; 16 x 1024, 512 blocks, 18.4, 20.8).
    pl.joined = pl.S > 1 && pl.S <= kMostJoined && n * pl.S <= 400;
    if (pl.joined) pl.ml = pl.total = 0;
    return pl;
}

PromptPlan plan_tiles(const kvi_attention &a, int32_t R, int32_t total_q, int32_t max_q, int32_t max_ctx)
{
    PromptPlan pl{};
    pl.tiles = true;
    const int per = 2 * tile_tokens(a.q_heads / a.kv_heads);
    // a request's last pair may be partly filled
    pl.chunks = std::max<int64_t>(1, std::min((int64_t)R * ((max_q + (int64_t)per - 1) / per), total_q / per + (int64_t)R));
    // a block for every SM
    const int64_t n = (int64_t)a.kv_heads * pl.chunks;
    plan_split(pl, a, part_rows(R, total_q, max_q), max_ctx, std::max<int64_t>(1, kPlanSms / n), kTilesAlone, 128);
    return pl;
}

// The tensor-core tiles want boxes of 8 tokens or more of a page and up to 128
// channels.  They take a fixed time for a call, and then hardly more for 128
// rows than for one; the other form pays by the row.  Measured, us, rows form
// and tiles (R requests, rows per KV head, keys): 8 KV heads of 128 channels,
// R = 1: 8 rows x 128 keys 6.4, 7.8, x 4096 11, 13; 16 rows x 128 keys 8.3, 7.8,
// x 4096 14, 13; R = 16: 8 rows x 4096 keys 61, 54.  2 KV heads of 64 channels,
// R = 16: 16 rows x 1024 keys 9.8, 11; 64 rows x 1024 keys 14, 12; few and short
// enough for one wave of the rows form, R = 1: 256 rows x 256 keys 7.7, 9.6.
bool tiles_fit(const kvi_attention &a, int32_t R, int32_t max_q, int32_t max_ctx, int32_t num_blocks, int32_t block_size)
{
    if (a.head_dim > 128 || block_size % 8 || num_blocks > (1 << 29)) return false;
    const int64_t rows = (int64_t)max_q * (a.q_heads / a.kv_heads);
    if (a.head_dim > 64) return rows > 8;
    return rows > 32 && (max_ctx > 256 || (int64_t)R * a.kv_heads * rows > 8192);
}

// Workspace for whichever form the cache's pages decide on, and for any smaller
// call: fewer rows are split into more pieces, so what a call needs does not go by
// its sizes, but pieces times blocks are bounded.  With n blocks before the split:
//   rows form: more than one piece only for n < kRowsWanted, and n S <= kRowsWanted
//   + n - 1 then; the rows of a block are 8 nt, of all KV heads together;
//   tiles: n S <= kPlanSms, and no more than `per` tokens of G heads a block.
// Also no row has more pieces than there are 128 keys.
size_t prompt_bytes(const kvi_attention &a, int32_t R, int32_t total_q, int32_t max_q, int32_t max_ctx)
{
    const int64_t G = a.q_heads / a.kv_heads, rows = part_rows(R, total_q, max_q) * a.q_heads;
    const int64_t pieces = ((int64_t)max_ctx + 127) / 128;
    int64_t parts = max_ctx > kLongest ? 2 * rows : 0;
    auto at_most = [&](int64_t cap) { parts = std::max(parts, rows > cap ? cap : std::min(rows * pieces, cap)); };
    if (max_ctx > kRowsAlone) at_most(8 * (a.head_dim <= 128 && max_q * G > 8 ? 2 : 1) * (2 * kRowsWanted - 2));
    if (max_ctx > kTilesAlone && tiles_fit(a, R, max_q, max_ctx, 1, 8)) at_most(2 * tile_tokens((int)G) * G * kPlanSms);
    return std::max<size_t>(256, up256((size_t)parts * a.head_dim * 4) + up256((size_t)parts * 8));
}

template <int DP, int NT, bool JOINED>
cudaError_t run_rows_as(const PromptParams &p, int32_t R, cudaStream_t s)
{
    const int bytes = RowsSmem<DP, NT>::kBytes;
    const cudaError_t e = smem_opt_in(rows_kernel<DP, NT, JOINED>, bytes);
    if (e != cudaSuccess) return e;
    return launch_chained_clusters(rows_kernel<DP, NT, JOINED>, JOINED ? p.S : 1,
                                   dim3((unsigned)(p.S * p.chunks * p.H), (unsigned)R), kRowWarps * 32, bytes, s, p);
}

template <int DP, int NT>
cudaError_t run_rows(const PromptParams &p, int32_t R, cudaStream_t s)
{
    return p.joined ? run_rows_as<DP, NT, true>(p, R, s) : run_rows_as<DP, NT, false>(p, R, s);
}

cudaError_t launch_rows(const PromptParams &p, const PromptPlan &pl, int32_t R, cudaStream_t s)
{
    switch (pl.dp) {
    case 32: return pl.nt == 2 ? run_rows<32, 2>(p, R, s) : run_rows<32, 1>(p, R, s);
    case 64: return pl.nt == 2 ? run_rows<64, 2>(p, R, s) : run_rows<64, 1>(p, R, s);
    case 128: return pl.nt == 2 ? run_rows<128, 2>(p, R, s) : run_rows<128, 1>(p, R, s);
    default: return run_rows<256, 1>(p, R, s);
    }
}

bool sizes_ok(int32_t R, int32_t total_q, int32_t max_q, int32_t max_ctx)
{
    return R >= 1 && R <= KVI_MAX_REQUESTS && total_q >= 0 && max_q >= 0 && max_q <= total_q && max_ctx >= 0;
}

}  // namespace

}  // namespace kvi

using namespace kvi;

extern "C" size_t kvi_attn_prompt_workspace_bytes(const kvi_attention *a, int32_t R, int32_t total_q, int32_t max_q,
                                                  int32_t max_ctx)
{
    if (check_attention(a) != KVI_OK || !sizes_ok(R, total_q, max_q, max_ctx)) return 0;
    return prompt_bytes(*a, R, total_q, max_q, max_ctx);
}

extern "C" kvi_status kvi_attn_prompt(const kvi_attention *a, int32_t R, const void *d_q, int64_t q_row_stride,
                                      const int32_t *d_q_start, int32_t total_q, int32_t max_q,
                                      const int32_t *d_ctx_lens, int32_t max_ctx, const int32_t *d_block_tables,
                                      int32_t max_blocks, const kvi_paged_cache *cache, int32_t layer, void *d_out,
                                      int64_t out_row_stride, float *d_lse, void *d_ws, size_t ws_bytes,
                                      int32_t *d_status, kvi_stream_t stream)
{
    kvi_status st = check_attention(a);
    if (st != KVI_OK) return st;
    st = check_pages(cache, layer, R, max_blocks, d_block_tables);
    if (st != KVI_OK) return st;
    if (!sizes_ok(R, total_q, max_q, max_ctx))
        return arg_error("total_q=%d, max_q=%d (0..total_q) and max_ctx=%d must be >= 0", total_q, max_q, max_ctx);
    if (unusable(d_q_start, 4) || unusable(d_ctx_lens, 4) || unusable(d_status, 4) || (total_q && (!d_q || !d_out)) ||
        (d_lse && unusable(d_lse, 4)))
        return arg_error("a required pointer (q, q_start, ctx_lens, out, status) is NULL, or one is misaligned");
    const int64_t wide = (int64_t)a->q_heads * a->head_dim;
    if (reinterpret_cast<uintptr_t>(d_q) % 16 || reinterpret_cast<uintptr_t>(d_out) % 16 || q_row_stride % 8 ||
        out_row_stride % 8 || q_row_stride < wide || out_row_stride < wide)
        return arg_error("q and out rows must be 16-byte aligned, with strides of at least q_heads * head_dim elements");
    const PromptPlan pl = tiles_fit(*a, R, max_q, max_ctx, cache->num_blocks, cache->block_size)
                              ? plan_tiles(*a, R, total_q, max_q, max_ctx)
                              : plan_rows(*a, R, total_q, max_q, max_ctx);
    const size_t need = std::max<size_t>(256, pl.total);
    if (pl.chunks * pl.S * a->kv_heads > 0x7fffffff || (int64_t)max_q * (a->q_heads / a->kv_heads) > (1 << 30))
        return arg_error("max_q=%d is too large for this call", max_q);
    if (!d_ws || ws_bytes < need || reinterpret_cast<uintptr_t>(d_ws) % 256)
        return arg_error("workspace of %zu bytes (256-byte aligned) needed, %zu given", need, ws_bytes);
    uint8_t *ws = static_cast<uint8_t *>(d_ws);
    PromptParams p{};
    p.q = static_cast<const __nv_bfloat16 *>(d_q);
    p.q_stride = q_row_stride;
    p.q_start = d_q_start;
    p.R = R;
    p.total_q = total_q;
    p.max_q = max_q;
    p.per = tile_tokens(a->q_heads / a->kv_heads);
    p.ctx_lens = d_ctx_lens;
    p.max_ctx = max_ctx;
    p.max_blocks = max_blocks;
    p.block_tables = d_block_tables;
    p.num_blocks = cache->num_blocks;
    p.B = cache->block_size;
    p.H = a->kv_heads;
    p.Hq = a->q_heads;
    p.G = a->q_heads / a->kv_heads;
    p.D = a->head_dim;
    p.pool = static_cast<const __nv_bfloat16 *>(cache->layer_base[layer]);
    p.scale = a->scale * kLog2e;
    p.out = static_cast<__nv_bfloat16 *>(d_out);
    p.out_stride = out_row_stride;
    p.lse = d_lse;
    p.chunks = (int)pl.chunks;
    p.S = pl.S;
    p.span = pl.span;
    p.joined = pl.joined;
    p.by_request = total_q > (int64_t)R * max_q;
    p.po = reinterpret_cast<float *>(ws);
    p.ml = reinterpret_cast<float2 *>(ws + pl.ml);
    p.status = d_status;
    if (max_q == 0) return KVI_OK;  // no rows
    st = cuda_status(pl.tiles ? launch_tiles(p, stream) : launch_rows(p, pl, R, stream), "kvi_attn_prompt");
    if (st != KVI_OK || pl.S == 1 || pl.joined) return st;
    JoinParams j{};
    j.po = p.po;
    j.ml = p.ml;
    j.by_request = p.by_request;
    j.S = pl.S;
    j.span = pl.span;
    j.R = R;
    j.q_heads = a->q_heads;
    j.D = a->head_dim;
    j.q_start = d_q_start;
    j.total_q = total_q;
    j.max_q = max_q;
    j.ctx_lens = d_ctx_lens;
    j.max_ctx = max_ctx;
    j.max_blocks = max_blocks;
    j.block_size = cache->block_size;
    j.out = p.out;
    j.out_stride = out_row_stride;
    j.lse = d_lse;
    return cuda_status(launch_join(j, stream), "kvi_attn_prompt");
}
