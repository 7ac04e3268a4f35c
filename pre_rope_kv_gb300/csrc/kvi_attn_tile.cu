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
// where its own rounding to bf16 alone leaves 0.0017.  P as a sum of two bf16 numbers,
// which has room in tensor memory, leaves that too, and is not taken, as the second
// product twice and the softmax's part of it cost a quarter or more: 16 prompts with
// windows 106 us instead of 86, 8192 tokens 244 instead of 186, 64 users over a shared
// prefix 49 instead of 41, 24 questions 76 instead of 67.
// The two tiles alternate: while one tile's scores go through the softmax the
// tensor cores work on the other's products.  Two warps copy, K and V (a box per
// lane: a piece of a cache page, 64 channels wide), one looks over V where it has
// to be, one issues the matrix instructions, four per tile do the softmax.
//
// The running reference m moves only when a score passes it by 2^kLazy (O is
// rescaled in tensor memory then, which a row needs a few times in all).
// It may move at once: the matrix instructions run in the order of their issue
// and S of a tile is issued after the O of the tile before, so a tile's S
// being there means that its O is at rest.
//
// A row tile's last keys are often few: where no row sees the second half of them,
// its scores, weights and products are left out (37 tokens behind 1564 keys 14.8 to
// 14.2 us, windows 1%; not of a batch's shared prefix, which is whole tiles and
// took 3 us of 45 longer with it).
//
// Keys that only some rows see, or that lie past the end, are masked in S.
// Their values must not reach the output either (0 * inf is NaN), so in the
// few tiles that have such keys V is looked over in shared memory first: rows
// past the end become zero, and an infinity or NaN is replaced by zero and
// added, at the end, to the rows that see it.
//
// With a window a block walks over the first `sink` keys and those from its first
// row's window on, as if they lay one after the other; masks are a bit a column, so
// that they cost two instructions a score.  The keys that a batch shares are one
// request's, whose rows are all the batch's and see all of them; each piece's
// results go to the join.
//
// What bounds it: the matrix products (4 D flops per pair of row and key) for
// long prompts, and for ragged ones the 6 us or so that a block takes beside
// them (Q and the first keys, the rows' results), which nothing overlaps as a
// block fills its SM and its softmax warps store the results themselves.  32
// heads over 8 of 128 channels: one prompt of 8192 tokens 0.33 ms, 1670 TFLOP/s;
// 16 prompts of 1 to 2048 tokens and up to 1600 keys of memory 0.185 ms, 1150
// TFLOP/s; with windows of 2048 keys 0.186 ms for 8192 tokens (1.29 PFLOP/s), of 512
// for the 16 prompts 0.0856 ms (six tiles a block; 776 blocks are 5.1 for an SM, so
// that some SMs take six).  Of a block's 15 us there 3.2 pass until its first scores (request,
// block table, Q and K), 0.9 between the last P and O, 2.9 until the next block
// begins.  No faster: blocks that stay and take several pairs of tiles, the softmax
// warps storing the results all the same (0.35 and 0.19 ms), the pairs with the most
// keys first (0.34 and 0.195 ms), a barrier for each row tile's end; slower: two warps
// issuing matrix instructions, copies by cp.async instead of the tensor map, the
// first K before the first V.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "kvi_attn.cuh"
#include "kvi_sync.cuh"

namespace kvi {

namespace {

constexpr int kM = 128;           // rows of a tile, keys of a tile
constexpr int kCopyK = 8, kMmaWarp = 9, kCopyV = 10, kLookOver = 11;  // after four softmax warps per tile
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
    int32_t asked;          // V's tiles that have been asked for
    int32_t lost;           // a key's block lies outside the pool
    int32_t first[3][DP];   // first key whose value in a channel is +inf, -inf, NaN
    int32_t newest[3][DP];  // (windows) of the keys up to the block's first row, the last such
    int32_t part0;          // row of token 0 among the partial results
    int32_t skip, kept;     // (windows) keys left out, and the place from which on
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

// A warp looks over a tile of V before the products.  An infinity or NaN
// becomes zero, noted with its key for the rows that see it (a key past the end
// is seen by none).  The rule is that there is none: one maximum a word.
// With a window the rows that see a key are those from its position on, if that
// lies past the block's first row (`row0`), and else those whose window still
// reaches it: no window is shorter than a block's rows.  So of the former the
// first key says who sees any, of the latter the last (the first `sink` keys
// count as the latest of all).
template <int DP, int MODE>
__device__ __forceinline__ void check_values(uint8_t *v, int place0, TileTail<DP> &tl, int row0, int sink, int kept, int skip)
{
    constexpr int kChunks = TileSmem<DP>::kTile / 16;
    const int lane = threadIdx.x & 31;
    const uint4 *at = reinterpret_cast<const uint4 *>(v);
    // (four maxima, as each waits for the one before it)
    __nv_bfloat162 tops[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) tops[j] = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll 8
    for (int i = lane; i < kChunks; i += 32) {
        const uint4 x = at[i];
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) tops[j] = __hmax2_nan(tops[j], __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&w[j])));
    }
    tops[0] = __hmax2_nan(__hmax2_nan(tops[0], tops[1]), __hmax2_nan(tops[2], tops[3]));
    const uint32_t bits = *reinterpret_cast<const uint32_t *>(&tops[0]);
    const bool odd = (bits & 0x7f80u) == 0x7f80u || (bits & 0x7f800000u) == 0x7f800000u;
    if (!__any_sync(0xffffffffu, odd)) return;
    if (!tl.odd)
        for (int i = lane; i < 3 * DP; i += 32) {
            (&tl.first[0][0])[i] = INT32_MAX;
            if (MODE == kWindow) (&tl.newest[0][0])[i] = INT32_MIN;
        }
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
            const int place = place0 + row, key = MODE == kWindow && place >= kept ? place + skip : place;
            const int which = b == 0x7f80u ? 0 : b == 0xff80u ? 1 : 2, channel = 64 * half + 8 * chunk + k;
            if (MODE == kWindow && key <= row0)
                atomicMax(&tl.newest[which][channel], key < sink ? INT32_MAX : key);
            else
                atomicMin(&tl.first[which][channel], key);
            e[8 * i + k] = 0;
        }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
}

// Wait until a count in shared memory has reached `n`.
__device__ __forceinline__ bool wait_count(uint32_t count, int n, uint64_t limit_ns)
{
    uint64_t t0 = 0;
    for (uint32_t i = 0;; ++i) {
        int32_t have;
        asm volatile("ld.acquire.cta.shared.s32 %0, [%1];" : "=r"(have) : "r"(count) : "memory");
        if (have >= n) return true;
        if ((i & 31u) != 31u) continue;
        const uint64_t t = global_ns();
        if (t0 == 0) t0 = t;
        if (t - t0 > limit_ns) return false;
    }
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

// The lowest n bits (none below 0, all from 32 on)
__device__ __forceinline__ uint32_t low_bits(int n)
{
    uint32_t m;
    asm("bmsk.clamp.b32 %0, 0, %1;" : "=r"(m) : "r"(max(n, 0)));
    return m;
}

// Scores from column `vis` on are not seen.  A warp's rows are a few tokens, so few
// of its quarters of 32 columns are seen in part.
template <int COLS>
__device__ __forceinline__ void mask_scores(float *s, int vis)
{
#pragma unroll
    for (int q = 0; q < COLS; q += 32) {
        if (!__any_sync(0xffffffffu, vis < q + 32)) continue;
#pragma unroll
        for (int c = q; c < q + 32; ++c) s[c] = c < vis ? s[c] : neg_inf();
    }
}

// With a window: nor those that are past the first `sink` and below `low`; from
// column `kept` on a column's key is `skip` further.  (A bit a column: three
// comparisons each take a tile 1.6 us longer.)
template <int COLS>
__device__ __forceinline__ void mask_window(float *s, int vis, int sink, int low, int kept, int skip)
{
#pragma unroll
    for (int q = 0; q < COLS; q += 32) {
        const uint32_t near = low_bits(kept - q);
        const uint32_t first = low_bits(vis - q) & (~low_bits(low - q) | low_bits(sink - q));
        const uint32_t rest = low_bits(vis - skip - q) & ~low_bits(low - skip - q);
        const uint32_t seen = skip > 0 ? (first & near) | (rest & ~near) : first;
        if (__all_sync(0xffffffffu, seen == 0xffffffffu)) continue;
#pragma unroll
        for (int c = 0; c < 32; ++c) s[q + c] = (seen >> c) & 1u ? s[q + c] : neg_inf();
    }
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

template <int DP, int MODE>
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
        tl.asked = 0;
        tl.lost = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    // ---- the block's rows and keys
    const uint32_t rest = p.S == 1 ? blockIdx.x : blockIdx.x / (uint32_t)p.S;
    const int split = (int)(blockIdx.x - rest * (uint32_t)p.S);
    const int per = p.per;
    const bool flat = MODE == kShared && p.flat;
    wait_at_begin<MODE>(p);
    pdl_launch_dependents();
    // Blocks are for the tile pairs that there are, numbered request after request
    // and from a request's end (its heaviest) to its start; a warp looks over 32
    // requests at once.
    int item = (int)(rest / (uint32_t)p.H), r = -1, pair = 0;
    const int h = (int)(rest - (uint32_t)item * (uint32_t)p.H);
    RequestSpan rq{0, 0, 0};
    int part0 = 0;
    if (flat) {
        pair = item;
        r = batch_rows(p, rq);
        if (pair * 2 * per >= rq.n_q) return;
    }
    for (int r0 = 0; !flat && r0 < p.R; r0 += 32) {
        RequestSpan c{0, 0, 0};
        const bool asked = r0 + lane < p.R;
        int c_part0 = 0;
        const bool good = asked && (MODE == kShared
                                        ? request_past_prefix(r0 + lane, p.q_start, p.R, p.total_q, p.max_q, p.ctx_lens,
                                                              p.max_ctx, p.max_blocks, p.B, p.shared, c, c_part0)
                                        : request_span(r0 + lane, p.q_start, p.total_q, p.max_q, p.ctx_lens, p.max_ctx,
                                                       p.max_blocks, p.B, c) &&
                                              (MODE != kCausal || p.shared == 0 ||
                                               request_fits(c, p.q_start[0], p.q_start[p.R], p.R, p.total_q, p.max_q, p.shared)));
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
            if (MODE == kShared) part0 = __shfl_sync(0xffffffffu, c_part0, from_lane);
            break;
        }
        item -= __shfl_sync(0xffffffffu, sum, 31);
    }
    if (r < 0) {
        wait_at_end<MODE>(p);
        return;
    }
    const int tok0 = pair * 2 * per;  // the block's first token
    const int keys = MODE == kWindow ? min(rq.ctx, p.cap) : rq.ctx;  // that its pieces are for
    const bool whole = MODE != kShared && keys <= p.span;            // they are one piece
    if (split > 0 && (int64_t)split * p.span >= keys) {
        wait_at_end<MODE>(p);
        return;
    }
    const int seen0 = flat ? rq.ctx - 1 : rq.ctx - rq.n_q;  // last position that token 0 sees
    const int from = split * p.span;    // a multiple of 128
    // With a window a block's keys are the first `sink` ones and those from its first
    // window on, in whole boxes of the copies, one after the other: place u of them is
    // key u, or u + skip from place `kept` on, and tile j has the places from from + 128 j
    // on.  Boxes before that window (no row sees them) are not read.
    const int box_keys = kM >> box_shift;
    const int low = MODE == kWindow ? seen0 + tok0 - p.window + 1 : 0;
    int skip = 0, kept = 0;
    if (MODE == kWindow) {
        const uint32_t first = ((uint32_t)p.sink + box_keys - 1) & ~(uint32_t)(box_keys - 1);
        const uint32_t start = (uint32_t)max(0, low) & ~(uint32_t)(box_keys - 1);
        if (start > first) {
            // (the first keys fill up a tile of their own where sharing one saves none)
            const uint32_t own = (first + kM - 1) & ~(uint32_t)(kM - 1), rest = seen0 + min(rq.n_q, tok0 + 2 * per) - start;
            kept = (int)(start > own && (first + rest + kM - 1) / kM == (own + rest + kM - 1) / kM ? own : first);
            skip = (int)start - kept;
        }
    }
    auto key_at = [&](int u) { return MODE == kWindow && u >= kept ? u + skip : u; };
    // tiles of keys that each row tile walks over; token t sees up to seen0 + t
    // (indexed by constants alone: they stay in registers)
    int n_tiles[2];
    bool half_last[2];  // no row sees the second half of the last one
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t0 = tok0 + i * per, t1 = min(rq.n_q, t0 + per);
        const int seen = (flat ? rq.ctx : seen0 + t1) - skip;
        const int end = t0 < rq.n_q ? min(seen, from + p.span) : 0;
        n_tiles[i] = max(0, (end - from + kM - 1) / kM);
        half_last[i] = MODE != kShared && n_tiles[i] > 0 && end - from <= n_tiles[i] * kM - kM / 2;
    }
    const int n = max(n_tiles[0], n_tiles[1]);
    const int sure = seen0 + (flat ? 0 : tok0) + 1;  // keys below it are seen by every row
    // Tiles that some row sees in part: all from `first_partly` on; with a window also
    // those from `low_from` to `low_end`, past the first `sink` keys and before the
    // first key that every row's window holds.
    const int first_partly = sure - skip > from ? (sure - skip - from) / kM : 0;
    int low_from = 0, low_end = 0;
    if (MODE == kWindow) {
        const int held = seen0 + min(rq.n_q, tok0 + 2 * per) - p.window;
        low_from = max(0, p.sink / kM - from / kM);
        low_end = held <= 0 ? 0 : max(0, (held - skip - from + kM - 1) / kM);
    }
    auto partly = [&](int j) { return j >= first_partly || (MODE == kWindow && j >= low_from && j < low_end); };
    const int32_t *table = p.block_tables + (int64_t)r * p.max_blocks + (MODE == kShared && !flat ? p.shared / p.B : 0);

    // (below total_q; here, as r is not kept to the end)
    if (tid == 0) {
        tl.part0 = MODE == kShared ? part0 : p.by_request ? r * p.max_q : rq.q0;
        tl.skip = skip;
        tl.kept = kept;
    }

    // A tile of K (plane 0) or V (1) into a stage, a box a lane: 32 lanes cover
    // two halves of 16 boxes.  A piece past the end, or of a block that is not
    // there, reads as zeros from past a page's last token.
    const int half = lane >> box_shift, box = lane & ((1 << box_shift) - 1);
    // (Its block is asked for a tile ahead.)
    int at_token = 0, at_block = 0;
    auto wanted = [&](int key) {
        return key < rq.ctx && (MODE != kWindow || key + box_keys > low || key < p.sink);
    };
    auto block_of = [&](int j) {
        const int key = key_at(from + j * kM + box * box_keys);
        return wanted(key) ? table[(uint32_t)key / (uint32_t)p.B] : -1;
    };
    auto look_up = [&](int j, int block) {
        const int key = key_at(from + j * kM + box * box_keys);
        const bool there = (uint32_t)block < (uint32_t)p.num_blocks;
        // (noted before the copy is asked for, so before its scores are looked at)
        if (warp == kCopyK && __any_sync(0xffffffffu, wanted(key) && !there) && lane == 0) {
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
        for (int j = 0; j < n; ++j) {
            look_up(j, block);
            if (j + 1 < n) block = block_of(j + 1);
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
            if (plane == 1 && lane == 0)
                asm volatile("st.release.cta.shared.s32 [%0], %1;" ::"r"(smem_u32(&tl.asked)), "r"(slots) : "memory");
        }
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
    } else if (warp == kLookOver) {
        // ------------------------------------------- values seen in part
        // (a warp of its own: the copies run ahead of it)
        for (int j = 0; j < n; ++j) {
            if (!partly(j)) continue;
            // V's copy is on its way (so its barrier is in this copy's phase, and stays there
            // until the products of this tile have been, which wait for this warp)
            bool got = wait_count(smem_u32(&tl.asked), j + 1, kTileWaitNs);
            const int slot = 2 * j + 1;  // (V's stages are the odd ones)
            got = got && mbar_wait_brisk(smem_u32(&tl.full[slot % Sm::kStages]), (uint32_t)((slot / Sm::kStages) & 1), kTileWaitNs);
            if (!__all_sync(0xffffffffu, got)) {
                if (lane == 0) record_status(p.status, KVI_ERR_TIMEOUT);
                break;
            }
            check_values<DP, MODE>(base + Sm::kRing + (slot % Sm::kStages) * Sm::kTile, from + j * kM, tl, sure - 1, p.sink,
                                   kept, skip);
            if (lane == 0) mbar_arrive(smem_u32(&tl.v_fixed[slot % Sm::kStages / 2]));
            __syncwarp();
        }
        __syncwarp();
        asm volatile("bar.arrive 1, 288;" ::: "memory");
    } else if (warp == kMmaWarp) {
        // -------------------------------------------------- matrix products
        if (n > 0) {
            const uint32_t lead = one_lane();
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            // This warp's latencies set the pace of everything here, so between two
            // products there is little more than a wait, and what the next tile of
            // keys needs is looked after while products are queued.
            constexpr uint32_t id_all = bf16_idesc(kM, false), id_half = bf16_idesc(kM / 2, false), id_o = bf16_idesc(DP, true);
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
            auto score_part = [&](int i, uint32_t stage, int k0, int k1, uint32_t id_s) {
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
            // the tile of each whose second half is left out
            const int h0 = half_last[0] ? n0 - 1 : -1, h1 = half_last[1] ? n1 - 1 : -1;
            uint32_t fixes = 0;  // the phase of each v_fixed, a bit a stage
            // Tile j of the keys, V in stage `vs` and K of j + 1 in stage `ks`; V's
            // copy has been waited for.
            auto step = [&](int j, uint32_t vs, uint32_t vnext, uint32_t ks, uint32_t kph, uint32_t vnph) {
                const uint32_t par = (uint32_t)(j & 1);
                const bool more0 = j + 1 < n0, more1 = j + 1 < n1, more = more0 || more1;
                if (partly(j)) {
                    if (!wait(fixed_bar + 4 * (vs - 1), (fixes >> vs) & 1u)) return false;
                    fixes ^= 1u << vs;
                }
                if (j < n0) {
                    if (!wait(p_bar, par)) return false;
                    values(0, vs, 0, j > 0);
                    if (more && !wait(full0 + 8 * ks, kph)) return false;
                    if (j != h0) {
                        if (!wait(p_bar + 8, par)) return false;
                        values(0, vs, 1, j > 0);
                    }
                    if (!more0) mma_commit(lead, o_bar);
                } else if (more && !wait(full0 + 8 * ks, kph)) {
                    return false;
                }
                if (more0) {
                    score_part(0, ks, 0, kSteps, j + 1 == h0 ? id_half : id_all);
                    mma_commit(lead, s_bar);
                }
                if (j < n1) {
                    if (!wait(p_bar + 16, par)) return false;
                    values(1, vs, 0, j > 0);
                    if (j != h1) {
                        if (!wait(p_bar + 24, par)) return false;
                        values(1, vs, 1, j > 0);
                    }
                    if (!more1) mma_commit(lead, o_bar + 8);
                }
                const uint32_t id1 = j + 1 == h1 ? id_half : id_all;
                if (more1) score_part(1, ks, 0, kSteps / 2, id1);
                mma_commit(lead, empty0 + 8 * vs);
                if (more && !wait(full0 + 8 * vnext, vnph)) return false;
                if (more1) {
                    score_part(1, ks, kSteps / 2, kSteps, id1);
                    mma_commit(lead, s_bar + 8);
                }
                if (more) mma_commit(lead, empty0 + 8 * ks);
                return true;
            };
            bool ok = wait(smem_u32(&tl.q_full), 0) && wait(full0, 0);
            if (ok) {
                if (n0 > 0) {
                    score_part(0, 0, 0, kSteps, h0 == 0 ? id_half : id_all);
                    mma_commit(lead, s_bar);
                }
                if (n1 > 0) {
                    score_part(1, 0, 0, kSteps, h1 == 0 ? id_half : id_all);
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
        const int last = seen0 + (flat ? 0 : token);
        float m = neg_inf(), limit = real ? neg_inf() : __int_as_float(0x7f800000), ref = 0.f, sum = 0.f;
        const float lazy = kLazy / p.scale;
        bool ok = true;
        auto soften = [&](auto cols, int j, bool in_part) {
            constexpr int kCols = decltype(cols)::value;  // that rows see any of
            // two loads of 64 scores; the first half's largest is found while the
            // second is on its way
            float s[kCols];
            tmem_load32(t_s, s);
            tmem_load32(t_s + 32, s + 32);
            tmem_wait_ld(s);
            tmem_wait_ld(s + 32);
            if constexpr (kCols == kM) {
                tmem_load32(t_s + 64, s + 64);
                tmem_load32(t_s + 96, s + 96);
            }
            float top;
            const bool lost = *reinterpret_cast<volatile int32_t *>(&tl.lost) != 0;
            if (in_part || lost) {
                if constexpr (kCols == kM) {
                    tmem_wait_ld(s + 64);
                    tmem_wait_ld(s + 96);
                }
                const int place0 = from + j * kM;
                if (MODE == kWindow)
                    mask_window<kCols>(s, last + 1 - place0, p.sink - place0, last - p.window + 1 - place0,
                                       tl.kept - place0, tl.skip);
                else
                    mask_scores<kCols>(s, last + 1 - place0);
                if (lost) {
                    uint32_t gone[4] = {0, 0, 0, 0};
                    for (int c = 0; c < kCols; ++c) {
                        const int key = place0 + c + (MODE == kWindow && place0 + c >= tl.kept ? tl.skip : 0);
                        if (key >= rq.ctx) break;
                        if ((uint32_t)table[key / p.B] >= (uint32_t)p.num_blocks) gone[c >> 5] |= 1u << (c & 31);
                    }
#pragma unroll
                    for (int c = 0; c < kCols; ++c)
                        if ((gone[c >> 5] >> (c & 31)) & 1u) s[c] = neg_inf();
                }
                top = largest64(s);
                if constexpr (kCols == kM) top = fmaxf(top, largest64(s + 64));
            } else {
                top = largest64(s);
                if constexpr (kCols == kM) {
                    tmem_wait_ld(s + 64);
                    tmem_wait_ld(s + 96);
                    top = fmaxf(top, largest64(s + 64));
                }
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
            for (int c = 0; c < kCols; c += 32) {
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
            announce(tl.p_full[i][kCols == kM ? 1 : 0]);
        };
        for (int j = 0; j < my; ++j) {
            const bool in_part = partly(j);
            ok = ok && mbar_wait_brisk(smem_u32(&tl.s_full[i]), (uint32_t)(j & 1), kTileWaitNs);
            if (!__all_sync(0xffffffffu, ok)) {
                if (lane == 0) record_status(p.status, KVI_ERR_TIMEOUT);
                ok = false;
                __syncwarp();
                break;
            }
            fence_after();
            if (MODE != kShared && j + 1 == my && (i ? half_last[1] : half_last[0]))
                soften(std::integral_constant<int, kM / 2>{}, j, in_part);
            else
                soften(std::integral_constant<int, kM>{}, j, in_part);
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
            const int parts = MODE == kShared ? p.parts : p.S, piece_no = MODE == kShared ? p.first + split : split;
            const float inv = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
            const bool odd = tl.odd != 0;
            // 32 channels of the row: asked for, and as they are to be
            auto ask_values = [&](int c, float *v) {
                if (my > 0) {
                    tmem_load32(t_o + c, v);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = 0.f;
                }
            };
            auto take_values = [&](int c, float *v) {
                if (odd) {
                    const float inf = __int_as_float(0x7f800000);
                    auto sees = [&](int which, int channel) {
                        return tl.first[which][channel] <= last ||
                               (MODE == kWindow && tl.newest[which][channel] > last - p.window);
                    };
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        if (sees(0, c + e)) v[e] += inf;
                        if (sees(1, c + e)) v[e] -= inf;
                        if (sees(2, c + e)) v[e] += inf - inf;
                    }
                    __syncwarp();
                }
            };
            auto row_values = [&](int c, float *v) {
                ask_values(c, v);
                tmem_wait_ld(v);
                take_values(c, v);
            };
            auto packed = [&](const float *v) {
                return make_uint4(pack_bf16(v[0] * inv, v[1] * inv), pack_bf16(v[2] * inv, v[3] * inv),
                                  pack_bf16(v[4] * inv, v[5] * inv), pack_bf16(v[6] * inv, v[7] * inv));
            };
            if (full) {
                uint8_t *to = base + Sm::kQ + i * Sm::kTile + row * 128;
                float both[2][32];  // (the next channels are on their way while these are stored)
                ask_values(0, both[0]);
#pragma unroll
                for (int c = 0; c < DP; c += 32) {
                    float *v = both[(c >> 5) & 1];
                    tmem_wait_ld(v);
                    if (c + 32 < DP) ask_values(c + 32, both[((c >> 5) + 1) & 1]);
                    take_values(c, v);
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
                          : static_cast<void *>(p.po + (part * parts + piece_no) * p.D));
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
                    p.ml[part * parts + piece_no] = make_float2(M, sum);
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
    wait_at_end<MODE>(p);
    fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

}  // namespace

template <int DP, int MODE>
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
    e = smem_opt_in(tile_kernel<DP, MODE>, bytes);
    if (e != cudaSuccess) return e;
    return launch_chained(tile_kernel<DP, MODE>, dim3((unsigned)(p.S * p.H * p.chunks)), kTileThreads, bytes, s, tq,
                          tkv, to, p, shift);
}

cudaError_t launch_tiles(const PromptParams &p, int mode, cudaStream_t s)
{
    if (mode == kWindow) return p.D <= 64 ? run_tiles<64, kWindow>(p, s) : run_tiles<128, kWindow>(p, s);
    if (mode == kShared) return p.D <= 64 ? run_tiles<64, kShared>(p, s) : run_tiles<128, kShared>(p, s);
    return p.D <= 64 ? run_tiles<64, kCausal>(p, s) : run_tiles<128, kCausal>(p, s);
}

}  // namespace kvi
