// kvi_attn_prompt.cu -- causal attention of packed prompts over the paged
// bf16 cache: row i of a request's n rows sees the positions <= ctx - n + i.
//
// A KV head's query rows are its group's heads for every token, token first:
// row = token * G + head, so the rows that read the same keys share a tile.
//
// Two more calls are forms of the same kernels: windows (kvi_attn_window; a row sees
// the last keys and the first ones, and tiles that no row of a block sees are left
// out) and batches with a shared prefix (kvi_attn_shared; the prefix is attended by
// all rows of the batch as one request's, beside each request's other keys, and the
// pieces joined).
//
// Long prompts run on the tensor cores' tiles (kvi_attn_tile.cu).  rows_kernel
// here takes 8 or 16 rows a block, for few rows and for the page and head sizes
// that the tiles do not take.  Its products are S^T = K Q^T (16 keys x 8 rows) and
// O^T = V^T P^T, as with few rows it is K and V that fill the matrix instruction's
// M.  Each warp streams its own tiles of 16 keys (16-byte asynchronous copies into
// a ring of its own, so no block-wide wait) and keeps a softmax of its own; the
// block's warps join at the end, and blocks that share a request's keys through one
// another's shared memory as a cluster, or in a second kernel.  Where a block's rows
// are all there are (decoding steps) the cache's bytes bound it: 64 requests x 1.5 k
// keys, 8 KV heads of 128 channels, 71 us, 5.3 TB/s; 64 windows of 1024 keys 51 us, 5.3
// TB/s; 64 users' 30 to 700 keys beside a prefix of 10240 for all 42 us.  (Slower: the
// keys of all requests in a row cut into as many chunks of one length as there are
// blocks at a time, 64 windows of 1024 keys 87 us and of 4096 keys 267 instead of 170:
// some SMs reach memory faster than others, and blocks that are handed out as they end
// leave those more.)
#include <cuda_runtime.h>

#include <algorithm>

#include "kvi_attn.cuh"

namespace kvi {

namespace {

// Warps of a block.  Three where a window's keys are long beside what a block takes
// to begin and end, so that four blocks fit an SM (64 windows of 1024 keys, 128
// channels, 54 us instead of 58.5, of 4096 keys 170 instead of 182, of 256 keys 26
// instead of 25; whole prefixes and their rests are as they were measured with four).
template <int DP, int MODE>
constexpr int kRowWarps = MODE == kWindow && DP == 128 ? 3 : 4;
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
template <int DP, int NT, int WARPS = 4>
struct RowsSmem {
    static constexpr int kPitch = DP * 2 + 16;
    static constexpr int kStage = 2 * 16 * kPitch;  // K then V of 16 keys
    static constexpr int kRing = kRowStages * kStage;
    static constexpr int kSum = WARPS * 8 * NT * (DP + 4) * 4;  // then the block's own
    static constexpr int kJoin = kSum + 8 * NT * DP * 4;
    static constexpr int kBytes = WARPS * kRing > kJoin ? WARPS * kRing : kJoin;
};

// DP: the head size rounded up to 32, 64, 128 or 256 (the rest reads as zero);
// 8 * NT rows per block.  JOINED: a chunk's pieces are a cluster, which joins them.
template <int DP, int NT, bool JOINED, int MODE>
__global__ void __launch_bounds__(kRowWarps<DP, MODE> * 32) rows_kernel(const __grid_constant__ PromptParams p)
{
    constexpr int kWarps = kRowWarps<DP, MODE>;
    using Sm = RowsSmem<DP, NT, kWarps>;
    constexpr int KS = DP / 16, CH = DP / 8;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ uint32_t s_here[kWarps][kRowStages];
    __shared__ float s_m[kWarps][8 * NT], s_l[kWarps][8 * NT];
    __shared__ float2 s_ml[8 * NT];  // of the block
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int split = blockIdx.x % p.S, chunk = (blockIdx.x / p.S) % p.chunks, h = blockIdx.x / p.S / p.chunks;
    int r = blockIdx.y;
    wait_at_begin<MODE>(p);
    pdl_launch_dependents();
    RequestSpan rq;
    int part0 = 0;
    const bool flat = MODE == kShared && p.flat;
    if (flat) {
        r = batch_rows(p, rq);
    } else if (MODE == kShared ? !request_past_prefix(r, p.q_start, p.R, p.total_q, p.max_q, p.ctx_lens, p.max_ctx,
                                                      p.max_blocks, p.B, p.shared, rq, part0)
                               : !request_span(r, p.q_start, p.total_q, p.max_q, p.ctx_lens, p.max_ctx, p.max_blocks, p.B, rq) ||
                                     (MODE == kCausal && p.shared &&
                                      !request_fits(rq, p.q_start[0], p.q_start[p.R], p.R, p.total_q, p.max_q, p.shared))) {
        if (tid == 0) record_status(p.status, KVI_ERR_OUT_OF_RANGE);
        wait_at_end<MODE>(p);
        return;
    }
    const int rows = rq.n_q * p.G, row0 = chunk * 8 * NT;
    if (row0 >= rows) {
        wait_at_end<MODE>(p);
        return;
    }
    const int pieces = max(1, ((MODE == kWindow ? min(rq.ctx, p.cap) : rq.ctx) + p.span - 1) / p.span);
    if (split >= pieces) {
        if (JOINED && pieces > 1) {  // (the others of the cluster count on it)
            cluster_sync();
            cluster_sync();
        }
        wait_at_end<MODE>(p);
        return;
    }
    const int seen_by_0 = flat ? rq.ctx - 1 : rq.ctx - rq.n_q;  // last position that token 0 sees
    int end = flat ? rq.ctx : min(rq.ctx, seen_by_0 + (min(rows, row0 + 8 * NT) - 1) / p.G + 1);
    // With a window the tiles of 16 keys are those of the first `sink` keys and
    // those from the block's first window on: tile i is tile i + skip of the keys
    // from `kept` on.
    // Keys before that window (no row sees them) are not read.
    const int low = MODE == kWindow ? seen_by_0 + row0 / p.G - p.window + 1 : 0;
    int skip = 0, kept = 0;
    if (MODE == kWindow) {
        const int start = max(0, low) / 16;
        kept = min(start, (int)(((int64_t)p.sink + 15) / 16));
        skip = start - kept;
        end -= skip * 16;
    }
    auto place_of = [&](int tile) { return MODE == kWindow && tile >= kept ? tile + skip : tile; };
    const int from = split * p.span, to = min(end, from + p.span);
    const bool whole = MODE != kShared && pieces == 1;

    // the rows' last visible positions: columns 2 t, 2 t + 1 of each n-tile
    int last[NT][2];
    int least = INT32_MAX;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int row = row0 + 8 * nt + 2 * t + c;
            last[nt][c] = row < rows ? seen_by_0 + (flat ? 0 : row / p.G) : -1;
            if (row < rows) least = min(least, last[nt][c]);
        }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
    // with a window: keys below it are not seen by the block's last row
    const int held = MODE == kWindow ? seen_by_0 + (min(rows, row0 + 8 * NT) - 1) / p.G - p.window + 1 : 0;
    auto sees = [&](int key, int upto) {
        return key <= upto && (MODE != kWindow || key > upto - p.window || key < p.sink);
    };

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
    // (of P's second numbers: an infinity among the values times a zero or less of them
    // must not make it a NaN, so that these are added to what is finite at the end)
    constexpr bool kTwoTerms = MODE == kWindow && NT == 1 && DP <= 128;
    float rest[kTwoTerms ? KS : 1][4];
#pragma unroll
    for (int i = 0; i < (kTwoTerms ? KS : 1); ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) rest[i][j] = 0.f;
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

    // ---- this warp's tiles: from / 16 + warp, + kWarps, ...
    uint8_t *ring = smem + warp * Sm::kRing;
    if (p.D < DP) {  // channels past D: copied never, zero for good
        for (int i = lane; i < kRowStages * 32; i += 32)
            for (int c = p.D / 8; c < CH; ++c)
                *reinterpret_cast<uint4 *>(ring + i * Sm::kPitch + c * 16) = make_uint4(0, 0, 0, 0);
    }
    const int32_t *table = p.block_tables + (int64_t)r * p.max_blocks + (MODE == kShared && !flat ? p.shared / p.B : 0);
    const int64_t plane = (int64_t)p.num_blocks * p.B * p.H * p.D;
    const int t0 = from / 16 + warp, t1 = (to + 15) / 16;
    const uint32_t ring_a = smem_addr(ring);

    auto wanted = [&](int key) { return key < rq.ctx && (MODE != kWindow || key >= low || key < p.sink); };
    // block of key `lane` (mod 16) of a tile; -1 outside
    auto block_of = [&](int tile) {
        const int key = place_of(tile) * 16 + (lane & 15);
        return tile < t1 && wanted(key) ? table[key / p.B] : -1;
    };
    auto issue = [&](int tile, int stage, int block) {
        const int key = place_of(tile) * 16 + (lane & 15);
        const bool asked = tile < t1 && wanted(key);
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
    for (int s = 0; s < kRowStages - 1; ++s) issue(t0 + s * kWarps, s, block_of(t0 + s * kWarps));
    int next_block = block_of(t0 + (kRowStages - 1) * kWarps);
    int stage = 0;
    for (int tile = t0; tile < t1; tile += kWarps) {
        const int ahead = tile + (kRowStages - 1) * kWarps;
        issue(ahead, stage == 0 ? kRowStages - 1 : stage - 1, next_block);
        next_block = block_of(ahead + kWarps);
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
        const int key0 = place_of(tile) * 16, key = key0 + g;
        const uint32_t here = s_here[warp][stage];
        bool move = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int kk = key + (i >> 1) * 8;
                const bool see = sees(kk, last[nt][i & 1]) && ((here >> (g + (i >> 1) * 8)) & 1u);
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
                    for (int i = 0; i < (kTwoTerms ? KS : 0); ++i) {
                        rest[i][c] *= f;
                        rest[i][c + 2] *= f;
                    }
#pragma unroll
                    for (int i = 0; i < KS; ++i) {
                        o[nt][i][c] *= f;
                        o[nt][i][c + 2] *= f;
                    }
                }
            __syncwarp();  // the next matrix instruction wants the warp as one
        }
        // ---- P in bf16 for the second product, whose operands are of one type and V's is
        // bf16.  Rounded once, each weight is up to 2^-8 of itself off, which leaves the
        // output 0.0023 off (mean square, of it) where its own rounding alone leaves
        // 0.0017.  Windows over few rows, which HBM bounds, take P as a sum of two bf16
        // numbers, 2^-16 of itself off at most, and are 0.0017 off (us, with two numbers
        // and one: 64 windows of 1024 keys, 128 channels 51.3, 50.7, 64 channels 29.7,
        // 32.1; 4 windows, 128 channels 12.1, 11.6).  The others do not: blocks of 16 rows, which issue bounds (16 prompts with
        // windows of 32 keys 329, 313), heads of 256 channels, whose sums then do not find
        // room (64 windows 106.7, 68.7), and the users' own keys beside a shared prefix,
        // whose tiles round P all the same (the output would be 0.0023 off with it too).  The
        // plain calls have one rounding, as their tiles.  The sum takes P unrounded.
        uint32_t b0[NT], b1[NT], r0 = 0, r1 = 0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float m0 = m[nt][0] == neg_inf() ? 0.f : m[nt][0], m1 = m[nt][1] == neg_inf() ? 0.f : m[nt][1];
            const float p0 = exp2_fast(s[nt][0] - m0), p1 = exp2_fast(s[nt][1] - m1);
            const float p2 = exp2_fast(s[nt][2] - m0), p3 = exp2_fast(s[nt][3] - m1);
            l[nt][0] += p0 + p2;
            l[nt][1] += p1 + p3;
            const uint32_t near0 = pack_bf16(p0, p1), near1 = pack_bf16(p2, p3);
            b0[nt] = transpose8x8(near0);
            b1[nt] = transpose8x8(near1);
            if (kTwoTerms) {
                r0 = transpose8x8(pack_bf16(p0 - bf16_lo(near0), p1 - bf16_hi(near0)));
                r1 = transpose8x8(pack_bf16(p2 - bf16_lo(near1), p3 - bf16_hi(near1)));
            }
        }
        // a tile that some row sees only in part: an infinity or NaN among its
        // values must not reach the rows that do not see it (0 * inf)
        const bool partly = key0 + 15 > least || (MODE == kWindow && key0 < held && key0 + 16 > p.sink);
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
                                    if (sees(key0 + kk, last[nt][c])) o[nt][i][2 * j + c] += x;
                        }
                    __syncwarp();
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816(o[nt][i], a[0], a[1], a[2], a[3], b0[nt], b1[nt]);
            if (kTwoTerms) mma16816(rest[kTwoTerms ? i : 0], a[0], a[1], a[2], a[3], r0, r1);
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
                float a = o[nt][i][c], b = o[nt][i][c + 2];
                if (kTwoTerms) {
                    if (fabsf(a) <= 3.4028235e38f) a += rest[kTwoTerms ? i : 0][c];
                    if (fabsf(b) <= 3.4028235e38f) b += rest[kTwoTerms ? i : 0][c + 2];
                }
                dst[16 * i] = a;
                dst[16 * i + 8] = b;
            }
        }
    __syncthreads();
    if (MODE == kShared && !flat && p.merges) {
        // ---- all of a row's keys past the prefix are here: its pieces are joined to them,
        // a row a warp, four channels a lane, eight pieces asked for before the sums
        pdl_wait();
        for (int n = warp; n < 8 * NT && row0 + n < rows; n += kWarps) {
            const int head = h * p.G + (row0 + n) % p.G, token = (row0 + n) / p.G;
            const int64_t part = (int64_t)(part0 + token) * p.Hq + head, at = (int64_t)(rq.q0 + token) * p.Hq + head;
            const float2 *ml = p.ml + part * p.parts;
            const float *po = p.po + part * p.parts * p.D;
            constexpr int kAhead = 8;
            float4 v[kAhead];
#pragma unroll
            for (int s = 0; s < kAhead; ++s)
                if (s < p.first && 4 * lane < p.D) v[s] = *reinterpret_cast<const float4 *>(po + s * p.D + 4 * lane);
            const float2 mine = lane < p.first ? ml[lane] : make_float2(neg_inf(), 0.f);  // of piece `lane`
            float M = mine.x;
            for (int s = lane + 32; s < p.first; s += 32) M = fmaxf(M, ml[s].x);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][n]);
            const float ref = M == neg_inf() ? 0.f : M, f0 = exp2_fast(mine.x - ref);
            float L = mine.y * f0, own[kWarps];
            for (int s = lane + 32; s < p.first; s += 32) L += ml[s].y * exp2_fast(ml[s].x - ref);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                own[w] = exp2_fast(s_m[w][n] - ref);
                L += s_l[w][n] * own[w];
            }
            const float inv = L == 0.f ? 0.f : 1.f / L;
            for (int d = 4 * lane; d - 4 * lane < p.D; d += 128) {
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                auto add = [&](const float4 &x, float f) {
                    acc.x = fmaf(f, x.x, acc.x);
                    acc.y = fmaf(f, x.y, acc.y);
                    acc.z = fmaf(f, x.z, acc.z);
                    acc.w = fmaf(f, x.w, acc.w);
                };
                if (d < p.D) {
#pragma unroll
                    for (int w = 0; w < kWarps; ++w)
                        add(*reinterpret_cast<const float4 *>(s_o + (w * 8 * NT + n) * kO + d), own[w]);
                }
                for (int b = 0; b < p.first; b += kAhead) {
                    if (b > 0 || d >= 128) {
#pragma unroll
                        for (int s = 0; s < kAhead; ++s)
                            if (b + s < p.first && d < p.D)
                                v[s] = *reinterpret_cast<const float4 *>(po + (int64_t)(b + s) * p.D + d);
                    }
#pragma unroll
                    for (int s = 0; s < kAhead; ++s) {
                        float f = __shfl_sync(0xffffffffu, f0, (b + s) & 31);
                        if (b + s >= 32) f = b + s < p.first ? exp2_fast(ml[b + s].x - ref) : 0.f;
                        // (a piece without a visible key adds nothing: its output may be anything)
                        if (b + s < p.first && d < p.D && f != 0.f) add(v[s], f);
                    }
                }
                if (d < p.D)
                    *reinterpret_cast<uint2 *>(p.out + (int64_t)(rq.q0 + token) * p.out_stride + (int64_t)head * p.D + d) =
                        make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
            }
            if (p.lse && lane == 0) p.lse[at] = L == 0.f ? neg_inf() : (M + log2f(L)) * kLn2;
        }
        return;
    }
    const int half = p.D / 2;
    for (int i = tid; i < 8 * NT * half; i += kWarps * 32) {
        const int n = i / half, d = (i % half) * 2, row = row0 + n;
        if (row >= rows) break;
        float M = neg_inf();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][n]);
        const float ref = M == neg_inf() ? 0.f : M;
        float L = 0.f;
        float2 acc = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
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
            const int64_t first_row = MODE == kShared ? part0 : p.by_request ? (int64_t)r * p.max_q : rq.q0;
            const int64_t part = (first_row + row / p.G) * p.Hq + head;
            const int parts = MODE == kShared ? p.parts : p.S, piece_no = MODE == kShared ? p.first + split : split;
            *reinterpret_cast<float2 *>(p.po + (part * parts + piece_no) * p.D + d) = acc;
            if (d == 0) p.ml[part * parts + piece_no] = make_float2(M, L);
        }
    }
    wait_at_end<MODE>(p);
    if (!JOINED || whole) return;
    // ---- each block of the cluster that has keys joins a part of the channels
    cluster_sync();
    for (int i = split * kWarps * 32 + tid; i < 8 * NT * half; i += pieces * kWarps * 32) {
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
int64_t most_parts(const kvi_attention &a, int32_t R, int64_t tokens, int32_t max_q, int32_t max_ctx)
{
    const int64_t G = a.q_heads / a.kv_heads, rows = tokens * a.q_heads;
    const int64_t pieces = ((int64_t)max_ctx + 127) / 128;
    int64_t parts = max_ctx > kLongest ? 2 * rows : 0;
    auto at_most = [&](int64_t cap) { parts = std::max(parts, rows > cap ? cap : std::min(rows * pieces, cap)); };
    if (max_ctx > kRowsAlone) at_most(8 * (a.head_dim <= 128 && max_q * G > 8 ? 2 : 1) * (2 * kRowsWanted - 2));
    if (max_ctx > kTilesAlone && tiles_fit(a, R, max_q, max_ctx, 1, 8)) at_most(2 * tile_tokens((int)G) * G * kPlanSms);
    return parts;
}

size_t part_bytes(const kvi_attention &a, int64_t parts)
{
    return std::max<size_t>(256, up256((size_t)parts * a.head_dim * 4) + up256((size_t)parts * 8));
}

size_t prompt_bytes(const kvi_attention &a, int32_t R, int32_t total_q, int32_t max_q, int32_t max_ctx)
{
    return part_bytes(a, most_parts(a, R, part_rows(R, total_q, max_q), max_q, max_ctx));
}

// The same of a batch with a shared prefix: its keys' pieces and the others', of
// which a row has one of each at least.
size_t shared_bytes(const kvi_attention &a, int32_t R, int32_t total_q, int32_t max_q, int32_t max_ctx, int32_t shared)
{
    const int64_t tokens = part_rows(R, total_q, max_q), rows = tokens * a.q_heads;
    return std::max(prompt_bytes(a, R, total_q, max_q, max_ctx),
                    part_bytes(a, std::max(rows, most_parts(a, 1, tokens, (int32_t)tokens, shared)) +
                                      std::max(rows, most_parts(a, R, tokens, max_q, max_ctx))));
}

template <int DP, int NT, bool JOINED, int MODE>
cudaError_t run_rows_as(const PromptParams &p, int32_t R, cudaStream_t s)
{
    const int bytes = RowsSmem<DP, NT, kRowWarps<DP, MODE>>::kBytes;
    const cudaError_t e = smem_opt_in(rows_kernel<DP, NT, JOINED, MODE>, bytes);
    if (e != cudaSuccess) return e;
    return launch_chained_clusters(rows_kernel<DP, NT, JOINED, MODE>, JOINED ? p.S : 1,
                                   dim3((unsigned)(p.S * p.chunks * p.H), (unsigned)R), kRowWarps<DP, MODE> * 32, bytes, s, p);
}

template <int DP, int NT, int MODE>
cudaError_t run_rows(const PromptParams &p, int32_t R, cudaStream_t s)
{
    if constexpr (MODE != kShared) {  // (whose pieces a second kernel joins)
        if (p.joined) return run_rows_as<DP, NT, true, MODE>(p, R, s);
    }
    return run_rows_as<DP, NT, false, MODE>(p, R, s);
}

template <int MODE>
cudaError_t launch_rows(const PromptParams &p, const PromptPlan &pl, int32_t R, cudaStream_t s)
{
    switch (pl.dp) {
    case 32: return pl.nt == 2 ? run_rows<32, 2, MODE>(p, R, s) : run_rows<32, 1, MODE>(p, R, s);
    case 64: return pl.nt == 2 ? run_rows<64, 2, MODE>(p, R, s) : run_rows<64, 1, MODE>(p, R, s);
    case 128: return pl.nt == 2 ? run_rows<128, 2, MODE>(p, R, s) : run_rows<128, 1, MODE>(p, R, s);
    default: return run_rows<256, 1, MODE>(p, R, s);
    }
}

cudaError_t launch_rows(const PromptParams &p, const PromptPlan &pl, int32_t R, int mode, cudaStream_t s)
{
    if (mode == kWindow) return launch_rows<kWindow>(p, pl, R, s);
    if (mode == kShared) return launch_rows<kShared>(p, pl, R, s);
    return launch_rows<kCausal>(p, pl, R, s);
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

namespace {

// The arguments that the calls on prompts share.
struct PromptCall {
    const char *name;
    const kvi_attention *a;
    int32_t R;
    const void *q;
    int64_t q_stride;
    const int32_t *q_start;
    int32_t total_q, max_q;
    const int32_t *ctx_lens;
    int32_t max_ctx;
    const int32_t *tables;
    int32_t max_blocks;
    const kvi_paged_cache *cache;
    int32_t layer;
    void *out;
    int64_t out_stride;
    float *lse;
    void *ws;
    size_t ws_bytes;
    int32_t *status;
    kvi_stream_t stream;
};

kvi_status check_prompt(const PromptCall &c)
{
    kvi_status st = check_attention(c.a);
    if (st != KVI_OK) return st;
    st = check_pages(c.cache, c.layer, c.R, c.max_blocks, c.tables);
    if (st != KVI_OK) return st;
    if (!sizes_ok(c.R, c.total_q, c.max_q, c.max_ctx))
        return arg_error("total_q=%d, max_q=%d (0..total_q) and max_ctx=%d must be >= 0", c.total_q, c.max_q, c.max_ctx);
    if (unusable(c.q_start, 4) || unusable(c.ctx_lens, 4) || unusable(c.status, 4) || (c.total_q && (!c.q || !c.out)) ||
        (c.lse && unusable(c.lse, 4)))
        return arg_error("a required pointer (q, q_start, ctx_lens, out, status) is NULL, or one is misaligned");
    const int64_t wide = (int64_t)c.a->q_heads * c.a->head_dim;
    if (reinterpret_cast<uintptr_t>(c.q) % 16 || reinterpret_cast<uintptr_t>(c.out) % 16 || c.q_stride % 8 ||
        c.out_stride % 8 || c.q_stride < wide || c.out_stride < wide)
        return arg_error("q and out rows must be 16-byte aligned, with strides of at least q_heads * head_dim elements");
    return KVI_OK;
}

kvi_status check_room(const PromptCall &c, int64_t blocks, int64_t rows, size_t need)
{
    if (blocks > 0x7fffffff || rows > (1 << 30)) return arg_error("max_q=%d is too large for this call", c.max_q);
    if (!c.ws || c.ws_bytes < need || reinterpret_cast<uintptr_t>(c.ws) % 256)
        return arg_error("workspace of %zu bytes (256-byte aligned) needed, %zu given", need, c.ws_bytes);
    return KVI_OK;
}

PromptParams params_of(const PromptCall &c, const PromptPlan &pl)
{
    PromptParams p{};
    p.q = static_cast<const __nv_bfloat16 *>(c.q);
    p.q_stride = c.q_stride;
    p.q_start = c.q_start;
    p.R = c.R;
    p.total_q = c.total_q;
    p.max_q = c.max_q;
    p.G = c.a->q_heads / c.a->kv_heads;
    p.per = tile_tokens(p.G);
    p.ctx_lens = c.ctx_lens;
    p.max_ctx = c.max_ctx;
    p.max_blocks = c.max_blocks;
    p.block_tables = c.tables;
    p.num_blocks = c.cache->num_blocks;
    p.B = c.cache->block_size;
    p.H = c.a->kv_heads;
    p.Hq = c.a->q_heads;
    p.D = c.a->head_dim;
    p.pool = static_cast<const __nv_bfloat16 *>(c.cache->layer_base[c.layer]);
    p.scale = c.a->scale * kLog2e;
    p.out = static_cast<__nv_bfloat16 *>(c.out);
    p.out_stride = c.out_stride;
    p.lse = c.lse;
    p.chunks = (int)pl.chunks;
    p.S = pl.S;
    p.span = pl.span;
    p.joined = pl.joined;
    p.by_request = c.total_q > (int64_t)c.R * c.max_q;
    p.po = static_cast<float *>(c.ws);
    p.status = c.status;
    return p;
}

JoinParams join_of(const PromptCall &c, const PromptParams &p)
{
    JoinParams j{};
    j.po = p.po;
    j.ml = p.ml;
    j.by_request = p.by_request;
    j.S = p.S;
    j.span = p.span;
    j.R = c.R;
    j.q_heads = p.Hq;
    j.D = p.D;
    j.q_start = c.q_start;
    j.total_q = c.total_q;
    j.max_q = c.max_q;
    j.ctx_lens = c.ctx_lens;
    j.max_ctx = c.max_ctx;
    j.max_blocks = c.max_blocks;
    j.block_size = p.B;
    j.out = p.out;
    j.out_stride = c.out_stride;
    j.lse = c.lse;
    return j;
}

cudaError_t launch_form(const PromptParams &p, const PromptPlan &pl, int32_t R, int mode, cudaStream_t s)
{
    return pl.tiles ? launch_tiles(p, mode, s) : launch_rows(p, pl, R, mode, s);
}

// Keys that the pieces of a row with a window cover at most: the blocks' tiles of
// `unit` keys from the first window of `tokens` tokens on, and the first ones.
int32_t window_cap(int32_t window, int32_t sink, int unit, int tokens)
{
    const int64_t cap = ((int64_t)sink + unit - 1) / unit * unit + window + tokens + 2 * unit;
    return (int32_t)std::min<int64_t>(cap, 0x7fffffff);
}

kvi_status attend_prompts(const PromptCall &c, int mode, int32_t window, int32_t sink, int32_t shared)
{
    const kvi_attention &a = *c.a;
    // The tiles' windows are no shorter than a block's rows, which check_values
    // counts on (shorter ones have few keys to a row, and suit the other form).
    const int tokens = 2 * tile_tokens(a.q_heads / a.kv_heads);
    const int32_t tile_cap = mode == kWindow ? window_cap(window, sink, 128, tokens) : 0x7fffffff;
    int32_t cap = tile_cap;
    PromptPlan pl{};
    if ((mode != kWindow || window >= tokens) &&
        tiles_fit(a, c.R, c.max_q, std::min(c.max_ctx, tile_cap), c.cache->num_blocks, c.cache->block_size)) {
        pl = plan_tiles(a, c.R, c.total_q, c.max_q, std::min(c.max_ctx, cap));
    } else {
        if (mode == kWindow) cap = window_cap(window, sink, 16, 16);
        const int32_t keys = std::min(c.max_ctx, cap);
        pl = plan_rows(a, c.R, c.total_q, c.max_q, keys);
        // Windows are of one length, so that blocks that find room at once end together:
        // one piece each where they are many, or the keys few (us, in pieces and in one,
        // 8 KV heads of 128 channels: 24 users x 1024 keys 24.9, 30.0; 40 x 1024 45.0, 35.9;
        // 64 x 1024 54.3, 50.1, x 256 26.1, 17.2, x 4096 170, 177; 16 x 256 13.0, 11.0; 8 x 256 9.0, 10.7).
        const int64_t n = (int64_t)c.R * a.kv_heads * pl.chunks;
        if (mode == kWindow && ((n >= 250 && keys <= 2560) || (n >= 96 && keys <= 384))) {
            pl.S = 1;
            pl.span = kLongest;
            pl.joined = false;
            pl.ml = pl.total = 0;
        }
    }
    kvi_status st = check_room(c, pl.chunks * pl.S * a.kv_heads, (int64_t)c.max_q * (a.q_heads / a.kv_heads),
                               std::max<size_t>(256, pl.total));
    if (st != KVI_OK || c.max_q == 0) return st;  // (or no rows)
    PromptParams p = params_of(c, pl);
    p.ml = reinterpret_cast<float2 *>(static_cast<uint8_t *>(c.ws) + pl.ml);
    p.window = window;
    p.sink = sink;
    p.cap = cap;
    p.shared = shared;
    st = cuda_status(launch_form(p, pl, c.R, mode, c.stream), c.name);
    if (st != KVI_OK || pl.S == 1 || pl.joined) return st;
    JoinParams j = join_of(c, p);
    j.cap = cap;
    j.shared = shared;
    return cuda_status(launch_join(j, c.stream), c.name);
}

// Whether the prefix is worth kernels of its own.  Not where a request's rows fill
// a block's two tiles by themselves, and so read it as often one way as the other
// (us, with and without; 8 KV heads of 4 heads of 128 channels, prefix 10240: 24
// requests x 37 tokens 67, 193; 8 x 37 58, 67; 4 x 64 51, 43; 16 x 128 274, 226),
// nor below 32 MB less to read, which cost what a launch and a join do (single
// tokens: 8 requests x 256 keys 12.0, 7.4; 4 x 1600, 20 MB, 13.3, 10.9; 16 x 512, 31
// MB, 14.4, 17.7; 2 x 10240, 42 MB, 19.1, 18.1; 64 x 256, 66 MB, 22.8, 25.8).  (Next to the
// limit bytes alone do not tell: 16 x 512 and 2 x 10240 go the slower way.)
bool shares(const kvi_attention &a, int32_t R, int64_t tokens, int32_t shared)
{
    const double less = ((double)R - 1) * shared * a.kv_heads * a.head_dim * 4;
    return tokens * (a.q_heads / a.kv_heads) < 256 * (int64_t)R && less >= (double)(32 << 20);
}

// The prefix in fewer pieces than there are SMs, so that the other keys are read on the
// rest of them meanwhile and a piece's fixed time is paid less often: as few as end with
// all the work shared out, at a block's 8 us and 1.33 a tile of 128 keys (of 128
// channels), and 35 KB a us of the others' keys for an SM, of which half of the most
// there can be are taken to be there.  Not below 5 of 12, as they may be fewer still (us,
// with a piece for every SM and so, single tokens; prefix 10240: 64 requests x 30 to 700
// keys 48.6, 41.1, 40 x 30 to 700 41.1, 32.7, 64 x 30 to 2000 79.6, 69.3, 400 x 10 to 60
// 103, 91; prefix 1600: 64 x 30 to 700 35.4, 32.4).
void share_out(PromptPlan &first, const kvi_attention &a, int32_t R, int32_t shared, int32_t own)
{
    const double units = (double)first.chunks * a.kv_heads, tiles = 1.33 * ((shared + 127) / 128);
    const double others = (double)R * own / 2 * a.kv_heads * a.head_dim * 4 / 35e3;
    int S = (5 * first.S + 11) / 12;
    while (S < first.S && 8 + tiles / S > (units * (8 * S + tiles) + others) / kPlanSms) ++S;
    const int64_t span = ((int64_t)shared + S - 1) / S;
    first.span = (int)std::max<int64_t>(first.span, std::min<int64_t>((span + 127) / 128 * 128, kLongest));
    first.S = (int)(((int64_t)shared + first.span - 1) / first.span);
}

kvi_status attend_shared(const PromptCall &c, int32_t shared)
{
    const kvi_attention &a = *c.a;
    const int32_t blocks = c.cache->num_blocks, B = c.cache->block_size, own = c.max_ctx - shared;
    const int64_t tokens = part_rows(c.R, c.total_q, c.max_q), rows = tokens * a.q_heads;
    const int32_t all = (int32_t)tokens;
    PromptPlan first = tiles_fit(a, 1, all, shared, blocks, B) ? plan_tiles(a, 1, all, all, shared)
                                                               : plan_rows(a, 1, all, all, shared);
    // Few rows take the rows form, which reads the keys beside the prefix's tiles, several
    // blocks to an SM (us, tiles and rows; prefix 10240, own keys up to: 24 requests x 3
    // tokens, 900 48.9, 42.4, 2000 51.5, 44.6; 64 x 4, 2000 118, 94; 24 x 5, 100 42.3, 38.2,
    // x 8, 100 45.0, 43.9, 600 x 6 49.1, 52.5, 2000 x 8 61.9, 70.1).
    const int64_t most = (int64_t)c.max_q * (a.q_heads / a.kv_heads);
    const bool few = most <= 16 || (own <= 384 && most <= 32);
    PromptPlan rest = !few && tiles_fit(a, c.R, c.max_q, own, blocks, B) ? plan_tiles(a, c.R, c.total_q, c.max_q, own)
                                                                         : plan_rows(a, c.R, c.total_q, c.max_q, own);
    // Blocks that take a request's keys whole may join the prefix's pieces to them
    // themselves, without a third kernel, but hold their places until the prefix is done:
    // where they all have places at once (us, with a join and so, one token; prefix 1600:
    // 8 requests 14.3, 12.6, 16 17.0, 13.5, 24 21.9, 22.0, 32 19.2, 23.1; prefix 10240: 8
    // 21.6, 19.6, 24 29.6, 28.4, 48 33.0, 33.1; 10 x 4 tokens 26.7, 33.5).
    const bool merges = !rest.tiles && own <= 384 && most <= 8 && (int64_t)c.R * a.kv_heads * rest.chunks <= 200;
    if (merges) {
        rest.S = 1;
        rest.span = kLongest;
    } else if (first.tiles && !rest.tiles) {
        share_out(first, a, c.R, shared, own);
    }
    const int parts = first.S + (merges ? 0 : rest.S);
    const size_t ml = up256((size_t)rows * parts * a.head_dim * 4);
    kvi_status st = check_room(c, std::max(first.chunks * first.S, rest.chunks * rest.S) * a.kv_heads,
                               tokens * (a.q_heads / a.kv_heads),
                               std::max<size_t>(256, ml + up256((size_t)rows * parts * 8)));
    if (st != KVI_OK || c.max_q == 0) return st;
    PromptParams p = params_of(c, first);
    p.ml = reinterpret_cast<float2 *>(static_cast<uint8_t *>(c.ws) + ml);
    p.shared = shared;
    p.parts = parts;
    p.flat = 1;
    st = cuda_status(launch_form(p, first, 1, kShared, c.stream), c.name);
    if (st != KVI_OK) return st;
    p.flat = 0;
    p.first = first.S;
    p.chunks = (int)rest.chunks;
    p.S = rest.S;
    p.span = rest.span;
    p.joined = 0;
    p.merges = merges;
    st = cuda_status(launch_form(p, rest, c.R, kShared, c.stream), c.name);
    if (st != KVI_OK || merges) return st;
    JoinParams j = join_of(c, p);
    j.S = parts;
    j.first = first.S;
    j.shared = shared;
    return cuda_status(launch_join(j, c.stream), c.name);
}

}  // namespace

extern "C" kvi_status kvi_attn_prompt(const kvi_attention *a, int32_t R, const void *d_q, int64_t q_row_stride,
                                      const int32_t *d_q_start, int32_t total_q, int32_t max_q,
                                      const int32_t *d_ctx_lens, int32_t max_ctx, const int32_t *d_block_tables,
                                      int32_t max_blocks, const kvi_paged_cache *cache, int32_t layer, void *d_out,
                                      int64_t out_row_stride, float *d_lse, void *d_ws, size_t ws_bytes,
                                      int32_t *d_status, kvi_stream_t stream)
{
    const PromptCall c{"kvi_attn_prompt", a, R, d_q, q_row_stride, d_q_start, total_q, max_q, d_ctx_lens, max_ctx,
                       d_block_tables, max_blocks, cache, layer, d_out, out_row_stride, d_lse, d_ws, ws_bytes, d_status,
                       stream};
    const kvi_status st = check_prompt(c);
    return st != KVI_OK ? st : attend_prompts(c, kCausal, 0, 0, 0);
}

extern "C" kvi_status kvi_attn_window(const kvi_attention *a, int32_t R, const void *d_q, int64_t q_row_stride,
                                      const int32_t *d_q_start, int32_t total_q, int32_t max_q,
                                      const int32_t *d_ctx_lens, int32_t max_ctx, const int32_t *d_block_tables,
                                      int32_t max_blocks, const kvi_paged_cache *cache, int32_t layer, int32_t window,
                                      int32_t sink, void *d_out, int64_t out_row_stride, float *d_lse, void *d_ws,
                                      size_t ws_bytes, int32_t *d_status, kvi_stream_t stream)
{
    const PromptCall c{"kvi_attn_window", a, R, d_q, q_row_stride, d_q_start, total_q, max_q, d_ctx_lens, max_ctx,
                       d_block_tables, max_blocks, cache, layer, d_out, out_row_stride, d_lse, d_ws, ws_bytes, d_status,
                       stream};
    const kvi_status st = check_prompt(c);
    if (st != KVI_OK) return st;
    if (window < 1 || sink < 0) return arg_error("window=%d must be >= 1 and sink=%d >= 0", window, sink);
    if (window >= max_ctx || sink >= max_ctx) return attend_prompts(c, kCausal, 0, 0, 0);  // every row sees all before it
    if (window > (1 << 30)) return arg_error("window=%d is above 2^30", window);
    return attend_prompts(c, kWindow, window, sink, 0);
}

extern "C" size_t kvi_attn_shared_workspace_bytes(const kvi_attention *a, int32_t R, int32_t total_q, int32_t max_q,
                                                  int32_t max_ctx, int32_t shared)
{
    if (check_attention(a) != KVI_OK || !sizes_ok(R, total_q, max_q, max_ctx) || shared < 0) return 0;
    return shared_bytes(*a, R, total_q, max_q, max_ctx, std::min(shared, max_ctx));
}

extern "C" kvi_status kvi_attn_shared(const kvi_attention *a, int32_t R, const void *d_q, int64_t q_row_stride,
                                      const int32_t *d_q_start, int32_t total_q, int32_t max_q,
                                      const int32_t *d_ctx_lens, int32_t max_ctx, const int32_t *d_block_tables,
                                      int32_t max_blocks, const kvi_paged_cache *cache, int32_t layer, int32_t shared,
                                      void *d_out, int64_t out_row_stride, float *d_lse, void *d_ws, size_t ws_bytes,
                                      int32_t *d_status, kvi_stream_t stream)
{
    const PromptCall c{"kvi_attn_shared", a, R, d_q, q_row_stride, d_q_start, total_q, max_q, d_ctx_lens, max_ctx,
                       d_block_tables, max_blocks, cache, layer, d_out, out_row_stride, d_lse, d_ws, ws_bytes, d_status,
                       stream};
    const kvi_status st = check_prompt(c);
    if (st != KVI_OK) return st;
    if (shared < 0 || shared % cache->block_size || (int64_t)shared > (int64_t)max_blocks * cache->block_size ||
        (shared && shared >= max_ctx))
        return arg_error("shared=%d must be whole blocks of %d, fewer keys than max_ctx=%d and in the block tables", shared,
                         cache->block_size, max_ctx);
    const int64_t tokens = part_rows(R, total_q, max_q);
    return shared > 0 && shares(*a, R, tokens, shared) ? attend_shared(c, shared) : attend_prompts(c, kCausal, 0, 0, shared);
}
