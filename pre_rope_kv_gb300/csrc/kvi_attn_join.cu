// kvi_attn_join.cu -- the join of attention results computed in pieces of
// the keys, and the argument checks that the attention calls share.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "kvi_attn.cuh"

namespace kvi {

namespace {

// One warp per (query row, head): the pieces' (m, l) in one pass, then the
// weighted sum of their outputs.  Rows of a request with a single piece were
// written by the attention kernel itself.
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const __grid_constant__ JoinParams p)
{
    pdl_wait();
    pdl_launch_dependents();
    join_rows(p, blockIdx.x, blockIdx.y);
}

}  // namespace

cudaError_t launch_join(const JoinParams &p, cudaStream_t s)
{
    const int64_t rows = (int64_t)p.max_q * p.q_heads;
    return launch_chained(join_kernel, dim3((unsigned)((rows + kJoinWarps - 1) / kJoinWarps), (unsigned)p.R),
                          kJoinWarps * 32, 0, s, p);
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
