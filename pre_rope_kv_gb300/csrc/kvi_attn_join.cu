// kvi_attn_join.cu -- the join of attention results computed in pieces of
// the keys, and the argument checks that the attention calls share.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "kvi_attn.cuh"

namespace kvi {

namespace {

constexpr int kJoinWarps = 4;

// One warp per (query row, head): the pieces' (m, l) in one pass, then the
// weighted sum of their outputs.  Rows of a request with a single piece were
// written by the attention kernel itself.
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const JoinParams p)
{
    pdl_wait();
    const int r = blockIdx.y, lane = threadIdx.x & 31;
    RequestSpan q;
    if (!request_span(r, p.q_start, p.total_q, p.max_q, p.ctx_lens, p.max_ctx, p.max_blocks, p.block_size, q)) return;
    const int pieces = (q.ctx + p.span - 1) / p.span;
    if (pieces <= 1) return;
    const int64_t i = (int64_t)blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
    if (i >= (int64_t)q.n_q * p.q_heads) return;
    const int64_t row = (int64_t)q.q0 * p.q_heads + i;
    const float2 *ml = p.ml + row * p.S;
    float M = neg_inf();
    for (int s = lane; s < pieces; s += 32) M = fmaxf(M, ml[s].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float ref = M == neg_inf() ? 0.f : M;
    float L = 0.f;
    for (int s = lane; s < pieces; s += 32) L += ml[s].y * exp2_fast(ml[s].x - ref);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const float *po = p.po + row * p.S * p.D;
    __nv_bfloat16 *out = p.out + (row / p.q_heads) * p.out_stride + (row % p.q_heads) * p.D;
    for (int d = 2 * lane; d < p.D; d += 64) {
        float2 acc = make_float2(0.f, 0.f);
        for (int s = 0; s < pieces; ++s) {
            const float f = exp2_fast(ml[s].x - ref);
            const float2 v = *reinterpret_cast<const float2 *>(po + (int64_t)s * p.D + d);
            if (f != 0.f) {  // a piece without a visible key adds nothing
                acc.x = fmaf(f, v.x, acc.x);
                acc.y = fmaf(f, v.y, acc.y);
            }
        }
        *reinterpret_cast<uint32_t *>(out + d) = pack_bf16(acc.x * inv, acc.y * inv);
    }
    if (p.lse && lane == 0) p.lse[row] = L == 0.f ? neg_inf() : (M + log2f(L)) * kLn2;
}

}  // namespace

cudaError_t launch_join(const JoinParams &p, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    const int64_t rows = (int64_t)p.max_q * p.q_heads;
    cfg.gridDim = dim3((unsigned)((rows + kJoinWarps - 1) / kJoinWarps), (unsigned)p.R);
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, join_kernel, p);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

kvi_status arg_error(const char *fmt, ...)
{
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return set_error(KVI_ERR_INVALID_ARG, buf);
}

kvi_status cuda_status(cudaError_t e, const char *where)
{
    if (e == cudaSuccess) return KVI_OK;
    char buf[256];
    snprintf(buf, sizeof buf, "%s: %s", where, cudaGetErrorString(e));
    return set_error(KVI_ERR_CUDA, buf);
}

kvi_status check_attention(const kvi_attention *a)
{
    if (!a) return arg_error("attention is NULL");
    if (a->kv_heads < 1 || a->kv_heads > 4096 || a->q_heads < a->kv_heads || a->q_heads % a->kv_heads ||
        a->q_heads / a->kv_heads > KVI_MAX_ATTN_GROUP)
        return arg_error("q_heads=%d must be 1..%d times kv_heads=%d (1..4096)", a->q_heads, KVI_MAX_ATTN_GROUP,
                         a->kv_heads);
    if (a->head_dim < 16 || a->head_dim > KVI_MAX_ATTN_HEAD_DIM || a->head_dim % 16)
        return arg_error("head_dim=%d must be a multiple of 16 in [16, %d]", a->head_dim, KVI_MAX_ATTN_HEAD_DIM);
    if (!(a->scale > 0.f) || !std::isfinite(a->scale)) return arg_error("scale must be finite and > 0");
    return KVI_OK;
}

kvi_status check_pages(const kvi_paged_cache *c, int32_t layer, int32_t R, int32_t max_blocks, const void *block_tables)
{
    if (!c || !c->layer_base) return arg_error("cache or cache->layer_base is NULL");
    if (c->num_blocks < 1 || c->block_size < 1) return arg_error("num_blocks and block_size must be >= 1");
    if (layer < 0 || layer >= c->layers) return arg_error("layer=%d outside [0, %d)", layer, c->layers);
    if (!c->layer_base[layer] || reinterpret_cast<uintptr_t>(c->layer_base[layer]) % 16)
        return arg_error("layer_base[%d] is NULL or not 16-byte aligned", layer);
    if (R < 1 || R > KVI_MAX_REQUESTS) return arg_error("R=%d outside [1, %d]", R, KVI_MAX_REQUESTS);
    if (max_blocks < 1 || unusable(block_tables, 4)) return arg_error("block tables are required (max_blocks >= 1)");
    return KVI_OK;
}

}  // namespace kvi
