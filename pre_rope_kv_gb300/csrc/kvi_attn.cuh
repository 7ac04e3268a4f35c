// kvi_attn.cuh -- shared by the attention kernels (kvi_attn_prompt.cu,
// kvi_attn_decode4.cu) and the 4-bit cache (kvi_cache4.cu): the tensor-core
// and conversion helpers, the 4-bit page layout, and the join of partial
// results of work split over a long axis.  Not part of the public ABI.
//
// Softmax in pieces.  With s_p = scale <q, k_p> in units of log2 (scale
// times log2 e), a piece of the keys is summed up by (m, l, o): m a number no
// smaller than max s_p - kLazy, l = sum 2^(s_p - m) and o = sum 2^(s_p - m)
// v_p, all float32.  Pieces join by M = max m: l = sum l_i 2^(m_i - M), o
// likewise; the output is o / l and the log of the sum (M + log2 l) ln 2.
// A piece no key of which is visible has m = -inf and l = 0, o = 0.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "kvi_internal.cuh"

namespace kvi {

constexpr int kPlanSms = 152;  // SMs that work is shared out over

// ------------------------------------------------------- 4-bit page layout
//
// One page holds B tokens (a multiple of 16) of one KV head: the codes of K
// and V, then their steps; G = D / 32 groups of 32 channels.  The order
// inside follows the matrix instruction's fragments, so that a lane's share
// of 16 tokens is a few wide loads and needs no shuffle:
//   K codes  [B][4][G] words: word (t, g) = channels 32 g + 8 t + n, nibble n
//   V codes  [B/2][8][G] words: word (s, g) = channels 32 g + 4 s + j of token
//            2 i (nibble j) and of token 2 i + 1 (nibble 4 + j)
//   K steps  [B][G] bf16            V steps  [B/2][G][2] bf16
// An element is step * (nibble - 8).
struct Page4 {
    int32_t B, D;
    __host__ __device__ int groups() const { return D / 32; }
    __host__ __device__ int64_t bytes() const { return (int64_t)B * D + (int64_t)B * groups() * 4; }
    __host__ __device__ int64_t v_codes() const { return (int64_t)B * D / 2; }
    __host__ __device__ int64_t k_steps() const { return (int64_t)B * D; }
    __host__ __device__ int64_t v_steps() const { return (int64_t)B * D + (int64_t)B * groups() * 2; }
};

// ------------------------------------------------------------------ joining

struct JoinParams {
    const float *po;         // [rows][S][D], the rows' order as PromptParams has it
    const float2 *ml;        // [rows][S] (m in log2 units, l)
    int32_t by_request;
    int32_t S, span;         // splits, keys per split
    int32_t cap = 0x7fffffff;  // keys that a row's pieces cover at most (windows)
    int32_t shared, first;   // leading keys that are in `first` pieces of their own
    int32_t R, q_heads, D;
    const int32_t *q_start;  // [R + 1] or null: one row per request
    int32_t total_q, max_q;
    const int32_t *ctx_lens;  // [R]
    int32_t max_ctx, max_blocks, block_size;
    __nv_bfloat16 *out;
    int64_t out_stride;
    float *lse;              // [total_q][q_heads] or null
};
cudaError_t launch_join(const JoinParams &p, cudaStream_t s);

// ------------------------------------------------------- attention of prompts

struct PromptParams {
    const __nv_bfloat16 *q;
    int64_t q_stride;
    const int32_t *q_start;
    int32_t R, total_q, max_q;
    const int32_t *ctx_lens;
    int32_t max_ctx, max_blocks;
    const int32_t *block_tables;
    int32_t num_blocks, B;
    int32_t H, Hq, G, D;
    const __nv_bfloat16 *pool;  // [2][num_blocks][B][H][D]
    float scale;                // times log2 e
    __nv_bfloat16 *out;
    int64_t out_stride;
    float *lse;
    int32_t chunks;             // row chunks per KV head: of each request, or (tiles) of all
    int32_t S, span;
    int32_t per;                // (tiles) tokens of a row tile
    int32_t joined;             // (rows) a chunk's pieces are a cluster, which joins them
    // (kWindow) the keys that a row sees, and how many of them a row's pieces cover at most
    int32_t window, sink, cap;
    // A batch whose requests share their first keys.  (kShared) flat: those keys, of all
    // rows as one request's; else each request's other keys.  Pieces from `first` on
    // of `parts` of a row.  merges: these keys are one piece, whose block joins the prefix's
    // pieces to it.
    int32_t shared, flat, first, parts, merges;
    // Partial results of row i of request r: at its place in q, or, where q has
    // more rows than R * max_q, at r * max_q + i; so they take no more of the
    // workspace than there can be rows that are split.
    int32_t by_request;
    float *po;
    float2 *ml;
    int32_t *status;
};

// The keys that a row at position i sees: i and all before it; those of the
// window (i - window, i] and the first `sink`; or (of a batch with a shared
// prefix) the prefix, or i and those before it from the prefix on.
enum : int { kCausal = 0, kWindow = 1, kShared = 2 };

// The tensor-core form (kvi_attn_tile.cu): two tiles of 128 rows a block.
// Tokens that a tile holds, and the launch (p.chunks: no fewer than the tile
// pairs of all requests together).
inline int tile_tokens(int G) { return 128 / G; }
cudaError_t launch_tiles(const PromptParams &p, int mode, cudaStream_t s);

// A tensor map of bf16 boxes with the 128-byte swizzle (rank <= 5; pitches in
// bytes of the dimensions past the first); out-of-range elements read as 0.
cudaError_t tensor_map_bf16(CUtensorMap *map, const void *ptr, int rank, const uint64_t *dims, const uint64_t *pitches,
                            const uint32_t *box);

// The checks of the attention calls' shared arguments (a message is recorded).
kvi_status check_attention(const kvi_attention *a);
kvi_status check_pages(const kvi_paged_cache *c, int32_t layer, int32_t R, int32_t max_blocks,
                       const void *block_tables);
kvi_status cache4_check(int32_t kv_heads, int32_t head_dim, const kvi_paged_cache *c, int32_t layer);
// Record the message as KVI_ERR_INVALID_ARG; a CUDA error as KVI_ERR_CUDA.
kvi_status arg_error(const char *fmt, ...);
// Whether a pointer is NULL or not aligned to `a` bytes.
inline bool unusable(const void *p, uintptr_t a) { return !p || reinterpret_cast<uintptr_t>(p) % a != 0; }
kvi_status cuda_status(cudaError_t e, const char *where);

#ifdef __CUDACC__

// Every kernel of these calls may begin while the previous kernel of the
// stream drains, waits for it before it touches memory (pdl_wait; the one kernel
// that does not is described at waits_last), and lets the next one begin
// (pdl_launch_dependents): what a launch costs is hidden behind the work before it.
// What they read may thus be written during their lifetime, so none of it goes
// through the read-only path (__ldg).  `blocks` > 1: the blocks along x form clusters
// of so many.
template <typename P, typename... Args>
inline cudaError_t launch_chained_clusters(void (*kernel)(P, Args...), int blocks, dim3 grid, dim3 block, size_t smem,
                                           cudaStream_t s, const std::decay_t<P> &p, const std::decay_t<Args> &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (blocks > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = (unsigned)blocks;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename P, typename... Args>
inline cudaError_t launch_chained(void (*kernel)(P, Args...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                                  const std::decay_t<P> &p, const std::decay_t<Args> &...args)
{
    return launch_chained_clusters(kernel, 1, grid, block, smem, s, p, args...);
}

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// The reference m of a running softmax moves only when a score passes it by
// more than 2^kLazy: sums and outputs then stay below 2^kLazy per key, far
// inside float32, and the accumulators are rescaled a few times per row
// instead of once per tile.
constexpr float kLazy = 8.0f;

constexpr int kMostJoined = 8;  // pieces that a cluster joins

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}

// What block `rank` of the cluster has at this address of its shared memory.
__device__ __forceinline__ float2 load_of_block(uint32_t addr, int rank)
{
    float2 v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %2, %3;\n\tld.shared::cluster.v2.f32 {%0, %1}, [a];\n\t}"
                 : "=f"(v.x), "=f"(v.y)
                 : "r"(addr), "r"(rank)
                 : "memory");
    return v;
}

__device__ __forceinline__ float neg_inf() { return __int_as_float((int)0xff800000u); }

// 2^x (the hardware's approximation, 2 ulp; -inf gives 0)
__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// D (16x8, float32) += A (16x16 bf16, row) B (16x8 bf16, col)
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same of f16 operands
__device__ __forceinline__ void mma16816_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                   uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// An 8x8 matrix of 16-bit elements (row = lane / 4, a pair of columns per
// lane) transposed across the warp.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b)
{
    const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&a),
                                     *reinterpret_cast<const __nv_bfloat162 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&v);
}

// The codes in nibbles 0 and 4 of w as two bf16 numbers (one and-or, one
// subtraction of 136)
__device__ __forceinline__ uint32_t codes_bf16x2(uint32_t w)
{
    uint32_t b;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(b) : "r"(w), "r"(0x000f000fu), "r"(0x43004300u));
    const uint32_t off = 0x43084308u;  // 136, 136
    const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&b),
                                     *reinterpret_cast<const __nv_bfloat162 *>(&off));
    return *reinterpret_cast<const uint32_t *>(&v);
}

// The codes in nibbles 0 and 4, and those in nibbles 1 and 5, of w as two f16
// numbers
__device__ __forceinline__ uint32_t codes_f16x2(uint32_t w)
{
    uint32_t b;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(b) : "r"(w), "r"(0x000f000fu), "r"(0x64006400u));
    const uint32_t off = 0x64086408u;  // 1032, 1032
    const __half2 v = __hsub2(*reinterpret_cast<const __half2 *>(&b), *reinterpret_cast<const __half2 *>(&off));
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t codes_f16x2_high(uint32_t w)
{
    uint32_t b;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(b) : "r"(w), "r"(0x00f000f0u), "r"(0x64006400u));
    const uint32_t part = 0x2c002c00u, off = 0xd480d480u;  // 1/16, -72
    const __half2 v = __hfma2(*reinterpret_cast<const __half2 *>(&b), *reinterpret_cast<const __half2 *>(&part),
                              *reinterpret_cast<const __half2 *>(&off));
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// (hi + lo) * s of two bf16 numbers each, lo no larger than hi's rounding: one
// rounding of the product to bf16 (lo * s rounds far below it)
__device__ __forceinline__ uint32_t scale_bf16x2(uint32_t hi, uint32_t lo, uint32_t s)
{
    const __nv_bfloat162 h = *reinterpret_cast<const __nv_bfloat162 *>(&hi);
    const __nv_bfloat162 l = *reinterpret_cast<const __nv_bfloat162 *>(&lo);
    const __nv_bfloat162 f = *reinterpret_cast<const __nv_bfloat162 *>(&s);
    const __nv_bfloat162 v = __hfma2(h, f, __hmul2(l, f));
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

}  // namespace

// A batch's own keys need nothing of the kernel before, which is that of its shared
// prefix: they begin beside it.  That this is in order:
//   - all blocks of the prefix's kernel wait for the work before it and only then let
//     this one begin, so that all of what that work wrote has been made visible to the
//     device by then; a fence takes the place of the wait here, so that nothing older is
//     read (24 questions 67.7 us, 66.6 without it, 64 users' tokens 41.9 and 41.6);
//   - blocks that join the prefix's pieces wait for its kernel first; of the others one
//     waits before it ends (early ends included), so that what follows, and waits for
//     this kernel, finds both done.  The rest make room (24 questions over 10240 keys
//     67.2 to 66.3 us, 32 users' tokens 34.3 to 32.7);
//   - a block that waits for the prefix's kernel holds up none of its blocks: they all
//     had their places before.
template <int MODE>
__device__ __forceinline__ bool waits_last(const PromptParams &p)
{
    return MODE == kShared && !p.flat;
}

template <int MODE>
__device__ __forceinline__ void wait_at_begin(const PromptParams &p)
{
    if (waits_last<MODE>(p))
        __threadfence();
    else
        pdl_wait();
}

template <int MODE>
__device__ __forceinline__ void wait_at_end(const PromptParams &p)
{
    if (waits_last<MODE>(p) && blockIdx.x == 0 && blockIdx.y == 0) pdl_wait();
}

// The rows and keys of request r, or false when its lengths are not usable.
struct RequestSpan {
    int32_t q0, n_q, ctx;
};
__device__ __forceinline__ bool request_span(int r, const int32_t *q_start, int total_q, int max_q,
                                             const int32_t *ctx_lens, int max_ctx, int max_blocks, int block_size,
                                             RequestSpan &o)
{
    o.q0 = q_start ? q_start[r] : r;
    const int q1 = q_start ? q_start[r + 1] : r + 1;
    o.ctx = ctx_lens[r];
    o.n_q = q1 - o.q0;
    return o.q0 >= 0 && q1 >= o.q0 && q1 <= total_q && o.n_q <= max_q && o.ctx >= 0 && o.ctx <= max_ctx &&
           (int64_t)o.ctx <= (int64_t)max_blocks * block_size;
}

// Whether a batch's rows, b0 = q_start[0] .. b1 = q_start[R] - 1, are rows of q, and no
// more than its requests can have.
__device__ __forceinline__ bool batch_fits(int b0, int b1, int R, int total_q, int max_q)
{
    return b0 >= 0 && b1 >= b0 && b1 <= total_q && (int64_t)b1 - b0 <= (int64_t)R * max_q;
}

// Whether a usable request is attended in a batch with a shared prefix: its rows are
// the batch's, and see all of the prefix.  The batch's rows are attended over the
// prefix as one request's, or not at all, so every kernel goes by this, those that
// read the prefix with each request's other keys included.
__device__ __forceinline__ bool request_fits(const RequestSpan &o, int b0, int b1, int R, int total_q, int max_q, int shared)
{
    return batch_fits(b0, b1, R, total_q, max_q) && o.q0 >= b0 && o.q0 + o.n_q <= b1 &&
           (o.n_q == 0 || o.ctx - o.n_q >= shared);
}

// The rows and keys of request r in a batch with a shared prefix: its keys past the
// prefix, and its first row's number in the batch.
__device__ __forceinline__ bool request_past_prefix(int r, const int32_t *q_start, int R, int total_q, int max_q,
                                                    const int32_t *ctx_lens, int max_ctx, int max_blocks,
                                                    int block_size, int shared, RequestSpan &o, int &part0)
{
    const int b0 = q_start[0], b1 = q_start[R];
    bool good = request_span(r, q_start, total_q, max_q, ctx_lens, max_ctx, max_blocks, block_size, o);
    good = good && request_fits(o, b0, b1, R, total_q, max_q, shared);
    part0 = good ? o.q0 - b0 : 0;
    o.ctx = max(0, o.ctx - shared);
    return good;
}

// The rows of all requests of a batch as one request's, over the shared prefix,
// which is read through the table of the first request that has rows (its
// number; without any, no rows).  Every warp for itself.
__device__ __forceinline__ int batch_rows(const PromptParams &p, RequestSpan &o)
{
    const int lane = threadIdx.x & 31, b0 = p.q_start[0], b1 = p.q_start[p.R];
    const bool good = batch_fits(b0, b1, p.R, p.total_q, p.max_q);
    o = RequestSpan{b0, good ? b1 - b0 : 0, p.shared};
    for (int r0 = 0; r0 < p.R; r0 += 32) {
        const int r = r0 + lane;
        const uint32_t some = __ballot_sync(0xffffffffu, r < p.R && p.q_start[r + 1] > p.q_start[r]);
        if (some) return r0 + __ffs((int)some) - 1;
    }
    o.n_q = 0;
    return 0;
}

namespace {

constexpr int kJoinWarps = 4;

// Block x of request r: its warps' (query row, head) rows.
__device__ __forceinline__ void join_rows(const JoinParams &p, int x, int r)
{
    const int lane = threadIdx.x & 31;
    RequestSpan q;
    int part0 = 0;
    if (p.first) {
        if (!request_past_prefix(r, p.q_start, p.R, p.total_q, p.max_q, p.ctx_lens, p.max_ctx, p.max_blocks, p.block_size,
                                 p.shared, q, part0))
            return;
    } else if (!request_span(r, p.q_start, p.total_q, p.max_q, p.ctx_lens, p.max_ctx, p.max_blocks, p.block_size, q) ||
               (p.shared && !request_fits(q, p.q_start[0], p.q_start[p.R], p.R, p.total_q, p.max_q, p.shared))) {
        return;
    }
    const int pieces = p.first + (min(q.ctx, p.cap) + p.span - 1) / p.span;
    if (pieces <= 1) return;
    const int64_t i = (int64_t)x * kJoinWarps + (threadIdx.x >> 5);
    if (i >= (int64_t)q.n_q * p.q_heads) return;
    const int64_t row = (int64_t)q.q0 * p.q_heads + i;
    const int64_t part = p.first        ? (int64_t)part0 * p.q_heads + i
                         : p.by_request ? (int64_t)r * p.max_q * p.q_heads + i
                                        : row;
    const float2 *ml = p.ml + part * p.S;
    const float *po = p.po + part * p.S * p.D;
    const int d0 = 4 * lane;
    // eight pieces' outputs are asked for before the sums are known
    constexpr int kAhead = 8;
    float4 v[kAhead];
#pragma unroll
    for (int s = 0; s < kAhead; ++s)
        if (s < pieces && d0 < p.D) v[s] = *reinterpret_cast<const float4 *>(po + (int64_t)s * p.D + d0);
    const float2 mine = lane < pieces ? ml[lane] : make_float2(neg_inf(), 0.f);  // of piece `lane`
    float M = mine.x;
    for (int s = lane + 32; s < pieces; s += 32) M = fmaxf(M, ml[s].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float ref = M == neg_inf() ? 0.f : M;
    const float f0 = exp2_fast(mine.x - ref);
    float L = mine.y * f0;
    for (int s = lane + 32; s < pieces; s += 32) L += ml[s].y * exp2_fast(ml[s].x - ref);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    const float inv = L == 0.f ? 0.f : 1.f / L;
    __nv_bfloat16 *out = p.out + (row / p.q_heads) * p.out_stride + (row % p.q_heads) * p.D;
    for (int d = d0; d - d0 < p.D; d += 128) {
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int b = 0; b < pieces; b += kAhead) {
            if (b > 0 || d > d0) {
#pragma unroll
                for (int s = 0; s < kAhead; ++s)
                    if (b + s < pieces && d < p.D) v[s] = *reinterpret_cast<const float4 *>(po + (int64_t)(b + s) * p.D + d);
            }
#pragma unroll
            for (int s = 0; s < kAhead; ++s) {
                float f = __shfl_sync(0xffffffffu, f0, (b + s) & 31);
                if (b + s >= 32) f = b + s < pieces ? exp2_fast(ml[b + s].x - ref) : 0.f;
                // a piece without a visible key adds nothing (its output may be anything)
                if (b + s < pieces && d < p.D && f != 0.f) {
                    acc.x = fmaf(f, v[s].x, acc.x);
                    acc.y = fmaf(f, v[s].y, acc.y);
                    acc.z = fmaf(f, v[s].z, acc.z);
                    acc.w = fmaf(f, v[s].w, acc.w);
                }
            }
        }
        if (d < p.D)
            *reinterpret_cast<uint2 *>(out + d) =
                make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    }
    if (p.lse && lane == 0) p.lse[row] = L == 0.f ? neg_inf() : (M + log2f(L)) * kLn2;
}

}  // namespace

#endif  // __CUDACC__

}  // namespace kvi
