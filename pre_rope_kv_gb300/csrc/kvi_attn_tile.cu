// kvi_attn_tile.cu -- causal attention of prompts on the 5th-generation tensor
// cores: the form of kvi_attn_prompt for long prompts.
//
// A block takes two tiles of up to 128 query rows of one request and KV head
// (row = token * G + head of the group, so that all heads that read the same
// keys share them) and walks over tiles of 128 keys:
//   S = Q K^T      tcgen05.mma, Q and K in shared memory, S in tensor memory
//   P = 2^(S - m)  a thread per row reads its 128 scores, keeps the running
//                  sum, and writes P in bf16 over S
//   O += P V       tcgen05.mma, P from tensor memory, V in shared memory
//                  as it lies in the cache (channels contiguous)
// P rounds to bf16, as the instruction takes both operands in one type and V is
// bf16; its sum takes it unrounded.  The output is 0.0023 off (mean square, of it),
// where its own rounding to bf16 alone leaves 0.0017.
// The two tiles alternate: while one tile's scores go through the softmax the
// tensor cores work on the other's products.  Two warps copy, K and V (a box per
// lane: a piece of a cache page, 64 channels wide), one issues the matrix
// instructions, four per tile do the softmax.
//
// The running reference m moves only when a score passes it by 2^kLazy (O is
// rescaled in tensor memory then, which a row needs a few times in all).
// It may move at once: the matrix instructions run in the order of their issue
// and S of a tile is issued after the O of the tile before, so a tile's S
// being there means that its O is at rest.
//
// Keys that only some rows see, or that lie past the end, are masked in S.
// Their values must not reach the output either (0 * inf is NaN), so in the
// few tiles that have such keys V is looked over in shared memory first: rows
// past the end become zero, and an infinity or NaN is replaced by zero and
// added, at the end, to the rows that see it.
//
// What bounds it: the matrix products (4 D flops per pair of row and key) for
// long prompts, and for ragged ones the 6 us or so that a block takes beside
// them (Q and the first keys, the rows' results), which nothing overlaps as a
// block fills its SM and its softmax warps store the results themselves.  32 heads over 8 of 128 channels: one prompt of 8192 tokens
// 0.33 ms, 1670 TFLOP/s; 16 prompts of 1 to 2048 tokens and up to 1600 keys of
// memory 0.19 ms, 1130 TFLOP/s.  No faster: blocks that stay and take several
// pairs of tiles, the softmax warps storing the results all the same (0.35 and
// 0.19 ms), the pairs with the most keys first (0.34 and
// 0.195 ms); slower: two warps issuing matrix instructions, copies by cp.async
// instead of the tensor map.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "kvi_attn.cuh"
#include "kvi_sync.cuh"

namespace kvi {

namespace {

constexpr int kM = 128;           // rows of a tile, keys of a tile
constexpr int kCopyK = 8, kMmaWarp = 9, kCopyV = 10;  // after four softmax warps per tile; one warp idles
constexpr int kTileThreads = 12 * 32;
// Registers: the launch gives 168 a thread (65536 / 384); the third warpgroup
// keeps 72 of them, so that the softmax's hold a row of scores: 2 * 216 + 72 =
// 3 * 168.
constexpr int kRegsSoft = 216, kRegsRest = 72;
constexpr uint64_t kTileWaitNs = 1000000000ull;
constexpr int kHalf = kM * 128;   // bytes of 128 rows of 64 channels

template <int DP>
struct TileSmem {
    static constexpr int kHalves = DP / 64;
    static constexpr int kTile = kHalves * kHalf;  // Q, K or V of 128 rows
    static constexpr int kStages = DP == 128 ? 4 : 6;
    static constexpr int kQ = 0, kRing = 2 * kTile, kTail = kRing + kStages * kTile;
};

template <int DP>
struct TileTail {
    uint64_t q_full;
    uint64_t full[TileSmem<DP>::kStages], empty[TileSmem<DP>::kStages];
    uint64_t s_full[2], p_full[2][2], o_full[2];  // p: P's first and second 64 keys
    uint64_t v_fixed[TileSmem<DP>::kStages / 2];  // of V's stages
    uint64_t drained;
    uint32_t tmem;
    int32_t odd;            // `first` holds something
    int32_t lost;           // a key's block lies outside the pool
    int32_t first[3][DP];   // first key whose value in a channel is +inf, -inf, NaN
    int32_t part0;          // row of token 0 among the partial results
};

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory descriptors, 128-byte swizzle: rows of 128 bytes in groups of
// 8 (1024 bytes).  K-major (Q, K): the stride offset is the group's; MN-major
// (V): 64 channels of 8 keys are a group, the next 64 channels lie a half on
// (the leading offset, which K-major operands do not use).  The address is the
// low word's, in units of 16 bytes, so that a step is an addition to it.
constexpr uint32_t kDescHi = (1024 >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t a) { return (a >> 4) | ((uint32_t)(kHalf >> 4) << 16); }
__device__ __forceinline__ uint64_t desc(uint32_t lo) { return ((uint64_t)kDescHi << 32) | lo; }

// Instruction descriptor: D float32, A and B bf16, M = 128, N, B K- or MN-major
__host__ __device__ constexpr uint32_t bf16_idesc(int n, bool b_mn)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(kM >> 4) << 24);
}

// The matrix instructions are issued by one lane but reached by the whole warp:
// their operands then are uniform values, which is where the instruction takes
// them from.
__device__ __forceinline__ uint32_t one_lane()
{
    uint32_t p;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p;
}

__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 q, %5, 0;\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
        "r"(add ? 1u : 0u), "r"(lead)
        : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 q, %5, 0;\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
        "r"(add ? 1u : 0u), "r"(lead)
        : "memory");
}

__device__ __forceinline__ void mma_commit(uint32_t lead, uint32_t bar)
{
    asm volatile(
        "{\n.reg .pred q;\nsetp.ne.b32 q, %1, 0;\n"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar), "r"(lead)
        : "memory");
}

// 32 columns of this warp's 32 lanes (no wait)
__device__ __forceinline__ void tmem_load32(uint32_t a, float *v)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,"
        "%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
          "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
          "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(a)
        : "memory");
}

__device__ __forceinline__ void tmem_store32(uint32_t a, const float *v)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"f"(v[0]),
        "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]), "f"(v[10]),
        "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]), "f"(v[16]), "f"(v[17]), "f"(v[18]), "f"(v[19]),
        "f"(v[20]), "f"(v[21]), "f"(v[22]), "f"(v[23]), "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]), "f"(v[28]),
        "f"(v[29]), "f"(v[30]), "f"(v[31]), "r"(a)
        : "memory");
}

__device__ __forceinline__ void tmem_store16(uint32_t a, const uint32_t *v)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(
            v[0]),
        "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
        "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(a)
        : "memory");
}

// Wait for this thread's loads; the registers are named so that nothing that
// uses them moves ahead of the wait.
__device__ __forceinline__ void tmem_wait_ld(float *v)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]),
                   "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]),
                   "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]),
                   "+f"(v[29]), "+f"(v[30]), "+f"(v[31])::"memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two float32 operations in one instruction
__device__ __forceinline__ uint64_t pair2(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ void split2(uint64_t v, float &a, float &b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ void box3(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void box4(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}

// from shared memory; what lies past the tensor's end is not written
__device__ __forceinline__ void box3_out(const CUtensorMap *map, int x, int y, int z, uint32_t src)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(z), "r"(src)
                 : "memory");
}

// The warp that copies V looks over a tile of it before the products.  An infinity or NaN
// becomes zero, noted with its key for the rows that see it (a key past the end
// is seen by none).  The rule is that there is none: one maximum a word.
template <int DP>
__device__ __forceinline__ void check_values(uint8_t *v, int key0, TileTail<DP> &tl)
{
    constexpr int kChunks = TileSmem<DP>::kTile / 16;
    const int lane = threadIdx.x & 31;
    const uint4 *at = reinterpret_cast<const uint4 *>(v);
    __nv_bfloat162 top = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll 4
    for (int i = lane; i < kChunks; i += 32) {
        const uint4 x = at[i];
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) top = __hmax2_nan(top, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&w[j])));
    }
    const uint32_t bits = *reinterpret_cast<const uint32_t *>(&top);
    const bool odd = (bits & 0x7f80u) == 0x7f80u || (bits & 0x7f800000u) == 0x7f800000u;
    if (!__any_sync(0xffffffffu, odd)) return;
    if (!tl.odd)
        for (int i = lane; i < 3 * DP; i += 32) (&tl.first[0][0])[i] = INT32_MAX;
    __syncwarp();
    if (lane == 0) tl.odd = 1;
    uint16_t *e = reinterpret_cast<uint16_t *>(v);
#pragma unroll 1
    for (int i = lane; odd && i < kChunks; i += 32) {
        const int half = i / (kHalf / 16), row = (i % (kHalf / 16)) / 8, chunk = (i & 7) ^ (row & 7);
#pragma unroll 1
        for (int k = 0; k < 8; ++k) {
            const uint32_t b = e[8 * i + k];
            if ((b & 0x7f80u) != 0x7f80u) continue;
            atomicMin(&tl.first[b == 0x7f80u ? 0 : b == 0xff80u ? 1 : 2][64 * half + 8 * chunk + k], key0 + row);
            e[8 * i + k] = 0;
        }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
}

// The largest of 64 scores
__device__ __forceinline__ float largest64(const float *s)
{
    float t[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) t[c] = max3(s[3 * c], s[3 * c + 1], s[3 * c + 2]);
#pragma unroll
    for (int c = 12; c + 8 <= 64; c += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] = max3(t[e], s[c + 2 * e], s[c + 2 * e + 1]);
    t[0] = max3(t[0], s[60], s[61]);
    t[1] = max3(t[1], s[62], s[63]);
    return fmaxf(max3(t[0], t[1], t[2]), t[3]);
}

// Scores from column `vis` on are not seen
__device__ __forceinline__ void mask_scores(float *s, int vis)
{
#pragma unroll
    for (int c = 0; c < kM; ++c) s[c] = c < vis ? s[c] : neg_inf();
}

// This warp's part of P has reached tensor memory.  (The arrival is lane 0's by a
// predicate, not a branch: what follows wants the warp as one.)
__device__ __forceinline__ void announce(uint64_t &bar)
{
    tmem_wait_st();
    fence_before();
    __syncwarp();
    asm volatile("{\n.reg .pred q;\nsetp.eq.u32 q, %1, 0;\n@q mbarrier.arrive.shared::cta.b64 _, [%0];\n}\n" ::"r"(
                     smem_u32(&bar)),
                 "r"(threadIdx.x & 31)
                 : "memory");
}

template <int DP>
__global__ void __launch_bounds__(kTileThreads, 1)
tile_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_kv,
            const __grid_constant__ CUtensorMap tm_out, const __grid_constant__ PromptParams p, int box_shift)
{
    using Sm = TileSmem<DP>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    TileTail<DP> &tl = *reinterpret_cast<TileTail<DP> *>(base + Sm::kTail);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (warp == kCopyK && lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_q)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_kv)) : "memory");
        mbar_init(smem_u32(&tl.q_full), 1);
        for (int s = 0; s < Sm::kStages; ++s) {
            mbar_init(smem_u32(&tl.full[s]), 1);
            mbar_init(smem_u32(&tl.empty[s]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&tl.s_full[i]), 1);
            mbar_init(smem_u32(&tl.p_full[i][0]), 4);
            mbar_init(smem_u32(&tl.p_full[i][1]), 4);
            mbar_init(smem_u32(&tl.o_full[i]), 1);
        }
        for (int s = 0; s < Sm::kStages / 2; ++s) mbar_init(smem_u32(&tl.v_fixed[s]), 1);
        mbar_init(smem_u32(&tl.drained), 1);
        tl.odd = 0;
        tl.lost = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    // ---- the block's rows and keys
    const uint32_t rest = p.S == 1 ? blockIdx.x : blockIdx.x / (uint32_t)p.S;
    const int split = (int)(blockIdx.x - rest * (uint32_t)p.S);
    const int per = p.per;
    pdl_wait();
    pdl_launch_dependents();
    // Blocks are for the tile pairs that there are, numbered request after request
    // and from a request's end (its heaviest) to its start; a warp looks over 32
    // requests at once.
    int item = (int)(rest / (uint32_t)p.H), r = -1, pair = 0;
    const int h = (int)(rest - (uint32_t)item * (uint32_t)p.H);
    RequestSpan rq{0, 0, 0};
    for (int r0 = 0; r0 < p.R; r0 += 32) {
        RequestSpan c{0, 0, 0};
        const bool asked = r0 + lane < p.R;
        const bool good = asked && request_span(r0 + lane, p.q_start, p.total_q, p.max_q, p.ctx_lens, p.max_ctx,
                                                p.max_blocks, p.B, c);
        if (asked && !good && h == 0 && split == 0 && warp == 0) record_status(p.status, KVI_ERR_OUT_OF_RANGE);
        const int pairs = good ? (c.n_q + 2 * per - 1) / (2 * per) : 0;
        int sum = pairs;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += u;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, sum > item);
        if (past) {
            const int from_lane = __ffs((int)past) - 1;
            pair = __shfl_sync(0xffffffffu, sum, from_lane) - 1 - item;
            r = r0 + from_lane;
            rq.q0 = __shfl_sync(0xffffffffu, c.q0, from_lane);
            rq.n_q = __shfl_sync(0xffffffffu, c.n_q, from_lane);
            rq.ctx = __shfl_sync(0xffffffffu, c.ctx, from_lane);
            break;
        }
        item -= __shfl_sync(0xffffffffu, sum, 31);
    }
    if (r < 0) return;
    const int tok0 = pair * 2 * per;  // the block's first token
    const bool whole = rq.ctx <= p.span;  // its keys are one piece
    if (split > 0 && (int64_t)split * p.span >= rq.ctx) return;
    const int seen0 = rq.ctx - rq.n_q;  // last position that token 0 sees
    const int from = split * p.span;    // a multiple of 128
    // tiles of keys that each row tile walks over; token t sees up to seen0 + t
    int n_tiles[2];  // (indexed by constants alone: they stay in registers)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t0 = tok0 + i * per, t1 = min(rq.n_q, t0 + per);
        const int end = t0 < rq.n_q ? min(seen0 + t1, from + p.span) : 0;
        n_tiles[i] = max(0, (end - from + kM - 1) / kM);
    }
    const int n = max(n_tiles[0], n_tiles[1]);
    const int sure = seen0 + tok0 + 1;  // keys below it are seen by every row
    const int32_t *table = p.block_tables + (int64_t)r * p.max_blocks;

    if (tid == 0) tl.part0 = p.by_request ? r * p.max_q : rq.q0;  // (below total_q; here, as r is not kept to the end)

    // A tile of K (plane 0) or V (1) into a stage, a box a lane: 32 lanes cover
    // two halves of 16 boxes.  A piece past the end, or of a block that is not
    // there, reads as zeros from past a page's last token.
    const int half = lane >> box_shift, box = lane & ((1 << box_shift) - 1), box_keys = kM >> box_shift;
    // (Its block is asked for a tile ahead.)
    int at_token = 0, at_block = 0;
    auto block_of = [&](int j) {
        const int key = from + j * kM + box * box_keys;
        return key < rq.ctx ? table[(uint32_t)key / (uint32_t)p.B] : -1;
    };
    auto look_up = [&](int j, int block) {
        const int key = from + j * kM + box * box_keys;
        const bool there = (uint32_t)block < (uint32_t)p.num_blocks;
        // (noted before the copy is asked for, so before its scores are looked at)
        if (warp == kCopyK && __any_sync(0xffffffffu, key < rq.ctx && !there) && lane == 0) {
            tl.lost = 1;
            record_status(p.status, KVI_ERR_OUT_OF_RANGE);
        }
        at_token = there ? key % (uint32_t)p.B : p.B;
        at_block = there ? block : 0;
    };
    auto copy_tile = [&](int plane, uint32_t stage) {
        const uint32_t bar = smem_u32(&tl.full[stage]);
        if (lane == 0) mbar_expect_tx(bar, Sm::kTile);
        __syncwarp();
        if (half < Sm::kHalves)
            box4(smem_u32(base + Sm::kRing) + stage * Sm::kTile + half * kHalf + box * box_keys * 128, &tm_kv, 64 * half, h,
                 at_token, plane * p.num_blocks + at_block, bar);
    };
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tl.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    __syncwarp();
    // The warp that copies K made the barriers and has nothing to wait for.  (A
    // barrier of its own: that warp may be at the last one before others are here.)
    fence_before();
    if (warp == kCopyK)
        asm volatile("bar.arrive 2, 384;" ::: "memory");
    else
        asm volatile("bar.sync 2, 384;" ::: "memory");
    fence_after();
    const uint32_t tmem = warp == kCopyK ? 0 : tl.tmem;
    // tensor memory: S (and P) of the two tiles, then their O
    constexpr int kColO = 2 * kM;

    if (warp >= kCopyK) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    if (warp == kCopyK || warp == kCopyV) {
        // ------------------------------------------------------------ copies
        // one warp copies Q and K, one V
        const int plane = warp == kCopyV ? 1 : 0;
        uint32_t stage = plane, phase = 1;  // an unused stage is empty
        bool ok = true;
        int slots = 0;
        int block = n > 0 ? block_of(0) : 0;
        if (plane == 0 && n > 0) {
            // rows past a tile's tokens keep what the memory held: their scores are
            // computed and not used
            const uint32_t bar = smem_u32(&tl.q_full);
            const int tiles = n_tiles[1] > 0 ? 2 : 1;
            if (lane == 0) mbar_expect_tx(bar, tiles * Sm::kHalves * per * p.G * 128);
            __syncwarp();
            if (lane < tiles * Sm::kHalves)
                box3(smem_u32(base + Sm::kQ) + (lane / Sm::kHalves) * Sm::kTile + (lane % Sm::kHalves) * kHalf, &tm_q,
                     64 * (lane % Sm::kHalves), h * p.G, rq.q0 + tok0 + (lane / Sm::kHalves) * per, bar);
        }
        // V of the tiles that some row sees in part is looked over before the next
        // V is asked for (it has been there for a while by then)
        const int first_partly = sure > from ? (sure - from) / kM : 0;
        auto look_over = [&](int j) {
            if (plane == 0 || j < first_partly) return true;
            const int slot = 2 * j + 1;  // (V's stages are the odd ones)
            const bool got = mbar_wait_brisk(smem_u32(&tl.full[slot % Sm::kStages]), (uint32_t)((slot / Sm::kStages) & 1), kTileWaitNs);
            if (!__all_sync(0xffffffffu, got)) {
                if (lane == 0) record_status(p.status, KVI_ERR_TIMEOUT);
                return false;
            }
            check_values<DP>(base + Sm::kRing + (slot % Sm::kStages) * Sm::kTile, from + j * kM, tl);
            if (lane == 0) mbar_arrive(smem_u32(&tl.v_fixed[slot % Sm::kStages / 2]));
            return true;
        };
        for (int j = 0; j < n; ++j) {
            look_up(j, block);
            if (j + 1 < n) block = block_of(j + 1);
            ok = j == 0 || look_over(j - 1);
            if (!ok) break;
            if (stage >= Sm::kStages) {
                stage = plane;
                phase ^= 1u;
            }
            bool got = true;
            if (lane == 0) got = mbar_wait_brisk(smem_u32(&tl.empty[stage]), phase, kTileWaitNs);
            if (!__shfl_sync(0xffffffffu, got ? 1 : 0, 0)) {
                if (lane == 0) record_status(p.status, KVI_ERR_TIMEOUT);
                ok = false;
                break;
            }
            copy_tile(plane, stage);
            ++slots;
            stage += 2;
        }
        if (ok && n > 0) ok = look_over(n - 1);
        // no copy may still be writing when the block ends
        if (!ok) {
            constexpr int kOwn = Sm::kStages / 2;
            if (lane < kOwn && lane < slots) {
                const int last = (slots - 1 - lane) / kOwn;
                (void)mbar_wait_brisk(smem_u32(&tl.full[2 * lane + plane]), (uint32_t)(last & 1), kTileWaitNs);
            }
            if (lane == 0 && plane == 0 && n > 0) (void)mbar_wait_brisk(smem_u32(&tl.q_full), 0, kTileWaitNs);
        }
        __syncwarp();
        if (plane == 1) asm volatile("bar.arrive 1, 288;" ::: "memory");
    } else if (warp == kMmaWarp) {
        // -------------------------------------------------- matrix products
        if (n > 0) {
            const uint32_t lead = one_lane();
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            // This warp's latencies set the pace of everything here, so between two
            // products there is little more than a wait, and what the next tile of
            // keys needs is looked after while products are queued.
            constexpr uint32_t id_s = bf16_idesc(kM, false), id_o = bf16_idesc(DP, true);
            constexpr uint32_t kTileLo = Sm::kTile >> 4;
            const uint32_t q_lo = desc_lo(smem_u32(base + Sm::kQ)), ring_lo = desc_lo(smem_u32(base + Sm::kRing));
            const uint32_t full0 = smem_u32(&tl.full[0]), empty0 = smem_u32(&tl.empty[0]);
            const uint32_t s_bar = smem_u32(&tl.s_full[0]), p_bar = smem_u32(&tl.p_full[0][0]);
            const uint32_t o_bar = smem_u32(&tl.o_full[0]), fixed_bar = smem_u32(&tl.v_fixed[0]);
            auto wait = [&](uint32_t bar, uint32_t parity) {
                const bool got = __all_sync(0xffffffffu, mbar_wait_brisk(bar, parity, kTileWaitNs));
                fence_after();
                return got;
            };
            auto score_part = [&](int i, uint32_t stage, int k0, int k1) {
#pragma unroll
                for (int k = k0; k < k1; ++k) {
                    const uint32_t at = ((k >> 2) * kHalf + (k & 3) * 32) >> 4;
                    mma_ss(lead, tm + i * kM, desc(q_lo + i * kTileLo + at), desc(ring_lo + stage * kTileLo + at), id_s, k > 0);
                }
            };
            constexpr int kSteps = DP / 16;
            // the keys of one half of a tile, as soon as their P is there
            auto values = [&](int i, uint32_t stage, int half, bool add) {
                const uint32_t b = ring_lo + stage * kTileLo + half * (kHalf / 2 >> 4);
#pragma unroll
                for (int k = 0; k < kM / 32; ++k)
                    mma_ts(lead, tm + kColO + i * DP, tm + i * kM + half * (kM / 4) + 8 * k, desc(b + k * (2048 >> 4)), id_o,
                           add || half > 0 || k > 0);
            };
            const int n0 = n_tiles[0], n1 = n_tiles[1];
            const int first_partly = sure > from ? (sure - from) / kM : 0;  // first tile that some row sees in part
            uint32_t fixes = 0;  // the phase of each v_fixed, a bit a stage
            // Tile j of the keys, V in stage `vs` and K of j + 1 in stage `ks`; V's
            // copy has been waited for.
            auto step = [&](int j, uint32_t vs, uint32_t vnext, uint32_t ks, uint32_t kph, uint32_t vnph) {
                const uint32_t par = (uint32_t)(j & 1);
                const bool more0 = j + 1 < n0, more1 = j + 1 < n1, more = more0 || more1;
                if (j >= first_partly) {
                    if (!wait(fixed_bar + 4 * (vs - 1), (fixes >> vs) & 1u)) return false;
                    fixes ^= 1u << vs;
                }
                if (j < n0) {
                    if (!wait(p_bar, par)) return false;
                    values(0, vs, 0, j > 0);
                    if (more && !wait(full0 + 8 * ks, kph)) return false;
                    if (!wait(p_bar + 8, par)) return false;
                    values(0, vs, 1, j > 0);
                    if (!more0) mma_commit(lead, o_bar);
                } else if (more && !wait(full0 + 8 * ks, kph)) {
                    return false;
                }
                if (more0) {
                    score_part(0, ks, 0, kSteps);
                    mma_commit(lead, s_bar);
                }
                if (j < n1) {
                    if (!wait(p_bar + 16, par)) return false;
                    values(1, vs, 0, j > 0);
                    if (!wait(p_bar + 24, par)) return false;
                    values(1, vs, 1, j > 0);
                    if (!more1) mma_commit(lead, o_bar + 8);
                }
                if (more1) score_part(1, ks, 0, kSteps / 2);
                mma_commit(lead, empty0 + 8 * vs);
                if (more && !wait(full0 + 8 * vnext, vnph)) return false;
                if (more1) {
                    score_part(1, ks, kSteps / 2, kSteps);
                    mma_commit(lead, s_bar + 8);
                }
                if (more) mma_commit(lead, empty0 + 8 * ks);
                return true;
            };
            bool ok = wait(smem_u32(&tl.q_full), 0) && wait(full0, 0);
            if (ok) {
                if (n0 > 0) {
                    score_part(0, 0, 0, kSteps);
                    mma_commit(lead, s_bar);
                }
                if (n1 > 0) {
                    score_part(1, 0, 0, kSteps);
                    mma_commit(lead, s_bar + 8);
                }
                mma_commit(lead, empty0);
                ok = wait(full0 + 8, 0);
            }
            // slots alternate K and V: V of tile j is slot 2 j + 1, K of j + 1 the next
            uint32_t vs = 1, ph = 0;
#pragma unroll 1
            for (int j = 0; j < n && ok; ++j) {
                const bool wraps = vs + 1 == Sm::kStages;
                const uint32_t ks = wraps ? 0 : vs + 1, vn = ks + 1, nph = wraps ? ph ^ 1u : ph;
                ok = step(j, vs, vn, ks, nph, nph);
                vs = vn;
                ph = nph;
            }
            if (!ok && lane == 0) record_status(p.status, KVI_ERR_TIMEOUT);
            // whatever ended the loop, no product may still run when tensor
            // memory is given back
            mma_commit(lead, smem_u32(&tl.drained));
            if (!wait(smem_u32(&tl.drained), 0) && lane == 0) record_status(p.status, KVI_ERR_TIMEOUT);
        }
        __syncwarp();
    }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
        // ----------------------------------------------------------- softmax
        const int i = warp >> 2, row = tid & (kM - 1);
        const int my = i ? n_tiles[1] : n_tiles[0];
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;  // this warp's part of tensor memory
        const uint32_t t_s = tmem + lanes + i * kM, t_o = tmem + lanes + kColO + i * DP;
        const int token = tok0 + i * per + row / p.G;
        const bool real = row < per * p.G && token < rq.n_q;
        const int last = seen0 + token;
        float m = neg_inf(), limit = real ? neg_inf() : __int_as_float(0x7f800000), ref = 0.f, sum = 0.f;
        const float lazy = kLazy / p.scale;
        bool ok = true;
        for (int j = 0; j < my; ++j) {
            const int key0 = from + j * kM;
            const bool partly = key0 + kM > sure;
            ok = ok && mbar_wait_brisk(smem_u32(&tl.s_full[i]), (uint32_t)(j & 1), kTileWaitNs);
            if (!__all_sync(0xffffffffu, ok)) {
                if (lane == 0) record_status(p.status, KVI_ERR_TIMEOUT);
                ok = false;
                __syncwarp();
                break;
            }
            fence_after();
            // two loads of 64 scores; the first half's largest is found while the
            // second is on its way
            float s[kM];
            tmem_load32(t_s, s);
            tmem_load32(t_s + 32, s + 32);
            tmem_wait_ld(s);
            tmem_wait_ld(s + 32);
            tmem_load32(t_s + 64, s + 64);
            tmem_load32(t_s + 96, s + 96);
            float top;
            const bool lost = *reinterpret_cast<volatile int32_t *>(&tl.lost) != 0;
            if (partly || lost) {
                tmem_wait_ld(s + 64);
                tmem_wait_ld(s + 96);
                mask_scores(s, last + 1 - key0);
                if (lost) {
                    uint32_t gone[4] = {0, 0, 0, 0};
                    for (int c = 0; c < kM && key0 + c < rq.ctx; ++c)
                        if ((uint32_t)table[(key0 + c) / p.B] >= (uint32_t)p.num_blocks) gone[c >> 5] |= 1u << (c & 31);
#pragma unroll
                    for (int c = 0; c < kM; ++c)
                        if ((gone[c >> 5] >> (c & 31)) & 1u) s[c] = neg_inf();
                }
                top = fmaxf(largest64(s), largest64(s + 64));
            } else {
                top = largest64(s);
                tmem_wait_ld(s + 64);
                tmem_wait_ld(s + 96);
                top = fmaxf(top, largest64(s + 64));
            }
            const bool move = top > limit;
            if (__any_sync(0xffffffffu, move)) {
                const float f = move ? exp2_fast((m - top) * p.scale) : 1.f;
                if (move) {
                    m = top;
                    limit = top + lazy;
                    ref = top * p.scale;
                    sum *= f;
                }
                __syncwarp();
                if (j > 0) {
#pragma unroll
                    for (int c = 0; c < DP; c += 32) {
                        float v[32];
                        tmem_load32(t_o + c, v);
                        tmem_wait_ld(v);
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] *= f;
                        tmem_store32(t_o + c, v);
                    }
                }
            }
            const uint64_t scale2 = pair2(p.scale, p.scale), ref2 = pair2(-ref, -ref);
            uint64_t part[2] = {0, 0};  // sums of even and odd keys, twice
#pragma unroll
            for (int c = 0; c < kM; c += 32) {
                uint32_t w[16];
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    float p0, p1;
                    split2(fma2(pair2(s[c + e], s[c + e + 1]), scale2, ref2), p0, p1);
                    p0 = exp2_fast(p0);
                    p1 = exp2_fast(p1);
                    part[(e >> 1) & 1] = add2(part[(e >> 1) & 1], pair2(p0, p1));
                    w[e / 2] = pack_bf16(p0, p1);
                }
                // the first half of P is announced when the third quarter is
                // computed, so that its way to tensor memory is not waited for
                if (c == 64) announce(tl.p_full[i][0]);
                tmem_store16(t_s + c / 2, w);
            }
            float a, b;
            split2(add2(part[0], part[1]), a, b);
            sum += a + b;
            announce(tl.p_full[i][1]);
        }
        // ---- the rows' results; the values have been looked over
        asm volatile("bar.sync 1, 288;" ::: "memory");
        if (n > 0 && ok) {
            // (without products of its own the tile's Q may still be on its way, and its
            // place is written to below)
            ok = mbar_wait_brisk(smem_u32(my > 0 ? &tl.o_full[i] : &tl.q_full), 0, kTileWaitNs);
            if (!__all_sync(0xffffffffu, ok)) {
                if (lane == 0) record_status(p.status, KVI_ERR_TIMEOUT);
                ok = false;
            }
            fence_after();
        }
        // One piece and all of a tile's tokens: its rows go out as Q came in, through
        // the tile's Q (which nothing reads any more), by a copy that a lane asks for.
        const bool full = whole && tok0 + (i + 1) * per <= rq.n_q;
        if (ok) {
            const int head = h * p.G + row % p.G;
            const int64_t tok = rq.q0 + token, at = tok * p.Hq + head;
            const int64_t part = ((int64_t)tl.part0 + token) * p.Hq + head;
            const float inv = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
            const bool odd = tl.odd != 0;
            // 32 channels of the row
            auto row_values = [&](int c, float *v) {
                if (my > 0) {
                    tmem_load32(t_o + c, v);
                    tmem_wait_ld(v);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = 0.f;
                }
                if (odd) {
                    const float inf = __int_as_float(0x7f800000);
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        if (tl.first[0][c + e] <= last) v[e] += inf;
                        if (tl.first[1][c + e] <= last) v[e] -= inf;
                        if (tl.first[2][c + e] <= last) v[e] += inf - inf;
                    }
                    __syncwarp();
                }
            };
            auto packed = [&](const float *v) {
                return make_uint4(pack_bf16(v[0] * inv, v[1] * inv), pack_bf16(v[2] * inv, v[3] * inv),
                                  pack_bf16(v[4] * inv, v[5] * inv), pack_bf16(v[6] * inv, v[7] * inv));
            };
            if (full) {
                uint8_t *to = base + Sm::kQ + i * Sm::kTile + row * 128;
#pragma unroll 1
                for (int c = 0; c < DP; c += 32) {
                    float v[32];
                    row_values(c, v);
#pragma unroll
                    for (int e = 0; e < 32; e += 8)
                        *reinterpret_cast<uint4 *>(to + (c >> 6) * kHalf + ((((c & 63) + e) / 8) ^ (row & 7)) * 16) = packed(v + e);
                }
            } else {
                // A thread holds a row, and rows lie far apart, so the warp's 32 rows go
                // through its quarter of the tile's Q (which nothing reads any more): row
                // by row out of it, a store covers whole lines.  16-byte pieces: 8
                // channels in bf16, or in two passes 4 in float32.
                constexpr int kPieces = DP / 8, kRowsAt = 32 / kPieces;
                uint4 *stage = reinterpret_cast<uint4 *>(base + Sm::kQ + i * Sm::kTile) + (warp & 3) * 32 * kPieces;
                const uint64_t mine = reinterpret_cast<uint64_t>(
                    whole ? static_cast<void *>(p.out + tok * p.out_stride + (int64_t)head * p.D)
                          : static_cast<void *>(p.po + (part * p.S + split) * p.D));
                const uint32_t rows_there = __ballot_sync(0xffffffffu, real);
#pragma unroll 1
                for (int pass = 0; pass < (whole ? 1 : 2); ++pass) {
                    const int c0 = whole ? 0 : pass * (DP / 2), c1 = whole ? DP : c0 + DP / 2;
#pragma unroll 1
                    for (int c = c0; c < c1; c += 32) {
                        float v[32];
                        row_values(c, v);
                        if (whole) {
#pragma unroll
                            for (int e = 0; e < 32; e += 8)
                                stage[lane * kPieces + (((c + e) / 8) ^ (lane & 7))] = packed(v + e);
                        } else {
#pragma unroll
                            for (int e = 0; e < 32; e += 4)
                                stage[lane * kPieces + (((c - c0 + e) / 4) ^ (lane & 7))] =
                                    make_uint4(__float_as_uint(v[e]), __float_as_uint(v[e + 1]), __float_as_uint(v[e + 2]),
                                               __float_as_uint(v[e + 3]));
                        }
                        __syncwarp();
                    }
                    const int piece = lane % kPieces;
                    const bool in_row = whole ? 8 * piece < p.D : c0 + 4 * piece < p.D;
#pragma unroll 4
                    for (int k = 0; k < 32; k += kRowsAt) {
                        const int rr = k + lane / kPieces;
                        const uint64_t to = __shfl_sync(0xffffffffu, mine, rr);
                        if (((rows_there >> rr) & 1u) && in_row)
                            reinterpret_cast<uint4 *>(to)[piece + pass * kPieces] = stage[rr * kPieces + (piece ^ (rr & 7))];
                    }
                    __syncwarp();
                }
            }
            if (real) {
                const float M = m * p.scale;
                if (!whole)
                    p.ml[part * p.S + split] = make_float2(M, sum);
                else if (p.lse)
                    p.lse[at] = sum == 0.f ? neg_inf() : (M + log2f(sum)) * kLn2;
            }
        }
        if (full) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            // (by every warp, whatever became of its waits)
            if (i == 0)
                asm volatile("bar.sync 3, 128;" ::: "memory");
            else
                asm volatile("bar.sync 4, 128;" ::: "memory");
            if ((warp & 3) == 0 && lane == 0 && ok) {
#pragma unroll
                for (int f = 0; f < Sm::kHalves; ++f)
                    box3_out(&tm_out, 64 * f, h * p.G, rq.q0 + tok0 + i * per, smem_u32(base + Sm::kQ + i * Sm::kTile + f * kHalf));
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            }
        }
    }
    fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

}  // namespace

template <int DP>
static cudaError_t run_tiles(const PromptParams &p, cudaStream_t s)
{
    CUtensorMap tq, tkv, to;
    const uint32_t per = (uint32_t)tile_tokens(p.G);
    const uint64_t qd[3] = {(uint64_t)p.D, (uint64_t)p.Hq, (uint64_t)p.total_q};
    const uint64_t qp[2] = {(uint64_t)p.D * 2, (uint64_t)p.q_stride * 2};
    const uint32_t qb[3] = {64, (uint32_t)p.G, per};
    cudaError_t e = tensor_map_bf16(&tq, p.q, 3, qd, qp, qb);
    if (e != cudaSuccess) return e;
    // K and V pieces: channels, heads, tokens of a page, pages (K's, then V's)
    int box = 8, shift = 4;  // 128 >> shift keys a box
    while (box < kM && p.B % (2 * box) == 0) {
        box *= 2;
        --shift;
    }
    const uint64_t row = (uint64_t)p.H * p.D * 2;
    const uint64_t kd[4] = {(uint64_t)p.D, (uint64_t)p.H, (uint64_t)p.B, 2 * (uint64_t)p.num_blocks};
    const uint64_t kp[3] = {(uint64_t)p.D * 2, row, row * p.B};
    const uint32_t kb[4] = {64, 1, (uint32_t)box, 1};
    e = tensor_map_bf16(&tkv, p.pool, 4, kd, kp, kb);
    if (e != cudaSuccess) return e;
    const uint64_t op[2] = {(uint64_t)p.D * 2, (uint64_t)p.out_stride * 2};
    e = tensor_map_bf16(&to, p.out, 3, qd, op, qb);
    if (e != cudaSuccess) return e;
    constexpr int bytes = TileSmem<DP>::kTail + (int)sizeof(TileTail<DP>) + 1024;
    static_assert(bytes <= 227 * 1024, "shared memory");
    e = smem_opt_in(tile_kernel<DP>, bytes);
    if (e != cudaSuccess) return e;
    return launch_chained(tile_kernel<DP>, dim3((unsigned)(p.S * p.H * p.chunks)), kTileThreads, bytes, s, tq,
                          tkv, to, p, shift);
}

cudaError_t launch_tiles(const PromptParams &p, cudaStream_t s)
{
    return p.D <= 64 ? run_tiles<64>(p, s) : run_tiles<128>(p, s);
}

}  // namespace kvi
