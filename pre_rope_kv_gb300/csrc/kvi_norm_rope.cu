// kvi_norm_rope.cu -- a step's own queries and keys: normalised per head,
// rotated to their positions (Section 5.1's rotation, under the conventions of
// kvi_rope) and, with the values, put into the paged cache (Section 3.4's
// scatter), in one pass.
//
//   y = x / sqrt(mean x^2 + eps) * w            (or y = x, without a weight)
//   out_i = y_i cos(p w_i) - y_j sin(p w_i),  out_j = y_j cos + y_i sin
//
// A warp takes a token's heads 32 / LPH at a time: LPH lanes hold a head, 16
// channels each (both elements of 8 pairs), so that the norm is a few shuffles
// and the rotation none.  A lane's 8 coefficient pairs serve all heads that its
// warp takes.  Squares are summed in float32, and y stays float32 until the one
// rounding of each result; the rotation is that of the injected keys, so without
// a weight a key gets the same bits as kvi_inject_paged gives it.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "kvi_attn.cuh"
#include "kvi_rotate.cuh"

namespace kvi {

namespace {

constexpr int kNormWarps = 4;

struct NormRopeParams {
    const __nv_bfloat16 *q, *k, *v, *wq, *wk;
    int64_t q_stride, k_stride, v_stride;
    __nv_bfloat16 *q_out, *k_out, *k_plain, *pool;
    int64_t q_out_stride, k_out_stride, k_plain_stride;
    int64_t plane;    // elements of the pool's K
    int64_t n_slots;
    const int64_t *slots;
    const int32_t *positions;
    int32_t max_position;
    const float4 *table;
    int64_t T;
    int32_t Hq, H, D;
    int32_t units_q, units_k, units;  // a token's: of q, of k, of all (v's last)
    int32_t warps;    // a token's
    float eps;
    int32_t *status;
};

__device__ __forceinline__ void unpack2(uint64_t v, float &a, float &b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}

// 16 channels as the rotation wants them: x0 the first elements of 8 pairs, x1
// the second ones, two to a word.
template <bool INTERLEAVED>
__device__ __forceinline__ void spread(const uint4 &a, const uint4 &b, uint64_t (&x0)[4], uint64_t (&x1)[4])
{
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (INTERLEAVED) {
            const uint32_t u = w[2 * i], v = w[2 * i + 1];
            x0[i] = f2(__uint_as_float(u << 16), __uint_as_float(v << 16));
            x1[i] = f2(__uint_as_float(u & 0xffff0000u), __uint_as_float(v & 0xffff0000u));
        } else {
            x0[i] = bf2_to_f2(w[i]);
            x1[i] = bf2_to_f2(w[4 + i]);
        }
    }
}

template <bool INTERLEAVED>
__device__ __forceinline__ void gather(const uint64_t (&x0)[4], const uint64_t (&x1)[4], uint4 &a, uint4 &b)
{
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (INTERLEAVED) {
            float p, q, r, s;
            unpack2(x0[i], p, q);
            unpack2(x1[i], r, s);
            w[2 * i] = bf16_pair(p, r);
            w[2 * i + 1] = bf16_pair(q, s);
        } else {
            w[i] = f2_to_bf2(x0[i]);
            w[4 + i] = f2_to_bf2(x1[i]);
        }
    }
    a = make_uint4(w[0], w[1], w[2], w[3]);
    b = make_uint4(w[4], w[5], w[6], w[7]);
}

// 1 / sqrt(mean x^2 + eps) of a head, which LPH lanes hold.
template <int LPH>
__device__ __forceinline__ float inverse_norm(const uint64_t (&x0)[4], const uint64_t (&x1)[4], int D, float eps)
{
    auto sum_of = [&](float f) {
        const uint64_t ff = f2(f, f);
        uint64_t s = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint64_t a = mul2(x0[i], ff), b = mul2(x1[i], ff);
            s = add2(s, add2(mul2(a, a), mul2(b, b)));
        }
        float lo, hi;
        unpack2(s, lo, hi);
        lo += hi;
#pragma unroll
        for (int o = 1; o < LPH; o <<= 1) lo += __shfl_xor_sync(0xffffffffu, lo, o);
        return lo;
    };
    float sum = sum_of(1.f), f = 1.f;
    // squares beyond float32: of values scaled down (eps is nothing beside them)
    const bool large = !(sum <= 3.0e38f);
    if (__any_sync(0xffffffffu, large)) {
        const float scaled = sum_of(0x1p-80f);
        if (large) {
            sum = scaled;
            f = 0x1p-80f;
            eps = 0.f;
        }
    }
    // (an infinity's or NaN's head is NaN throughout)
    return sum <= 3.0e38f ? f * rsqrtf(sum / (float)D + eps) : __int_as_float(0x7fffffff);
}

// NU: units (32 / LPH heads) of a warp
template <int LPH, bool INTERLEAVED, int NU>
__global__ void __launch_bounds__(kNormWarps * 32) norm_rope_kernel(const __grid_constant__ NormRopeParams p)
{
    constexpr int kHeads = 32 / LPH;
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * kNormWarps + (threadIdx.x >> 5);
    const int64_t t = w / p.warps;
    const int part = (int)(w - t * p.warps);
    pdl_wait();
    pdl_launch_dependents();
    if (t >= p.T) return;
    const int sub = lane / LPH, c = lane % LPH;
    // the lane's two pieces of 8 channels
    const int at0 = INTERLEAVED ? 16 * c : 8 * c, at1 = INTERLEAVED ? at0 + 8 : p.D / 2 + at0;
    const bool mine = 16 * c < p.D;

    uint4 a[NU], b[NU];
    int kind[NU], head[NU];  // 0 q, 1 k, 2 v, 3 nothing
#pragma unroll
    for (int i = 0; i < NU; ++i) {
        int u = part + i * p.warps;
        kind[i] = u >= p.units ? 3 : u < p.units_q ? 0 : u < p.units_q + p.units_k ? 1 : 2;
        if (kind[i] == 1) u -= p.units_q;
        if (kind[i] == 2) u -= p.units_q + p.units_k;
        head[i] = u * kHeads + sub;
        const __nv_bfloat16 *src = kind[i] == 0   ? p.q + t * p.q_stride
                                   : kind[i] == 1 ? p.k + t * p.k_stride
                                                  : p.v + t * p.v_stride;
        a[i] = b[i] = make_uint4(0, 0, 0, 0);
        if (kind[i] == 3 || !mine || head[i] >= (kind[i] == 0 ? p.Hq : p.H)) {
            head[i] = -1;
            continue;
        }
        src += (int64_t)head[i] * p.D;
        a[i] = *reinterpret_cast<const uint4 *>(src + at0);
        b[i] = *reinterpret_cast<const uint4 *>(src + at1);
    }
    const int32_t pos = p.positions[t];
    if (pos < 0 || pos >= p.max_position) {
        if (lane == 0) record_status(p.status, KVI_ERR_OUT_OF_RANGE);
        return;
    }
    int64_t slot = p.slots ? p.slots[t] : -1;
    if (slot >= p.n_slots) {
        if (lane == 0) record_status(p.status, KVI_ERR_OUT_OF_RANGE);
        slot = -1;
    }
    float4 cs[8];
    if (pos != 0 && mine) {
        const float4 *row = p.table + (int64_t)pos * (p.D / 2) + 8 * c;
#pragma unroll
        for (int e = 0; e < 8; ++e) cs[e] = __ldg(row + e);
    }
    auto put = [&](__nv_bfloat16 *dst, int h, const uint4 &x, const uint4 &y) {
        dst += (int64_t)h * p.D;
        *reinterpret_cast<uint4 *>(dst + at0) = x;
        *reinterpret_cast<uint4 *>(dst + at1) = y;
    };
    __nv_bfloat16 *page = slot < 0 ? nullptr : p.pool + slot * ((int64_t)p.H * p.D);
#pragma unroll
    for (int i = 0; i < NU; ++i) {
        if (kind[i] == 3) continue;
        const int h = head[i];
        if (kind[i] == 2) {
            if (h >= 0 && page) put(page + p.plane, h, a[i], b[i]);
            continue;
        }
        const __nv_bfloat16 *weight = kind[i] == 0 ? p.wq : p.wk;
        uint64_t x0[4], x1[4];
        spread<INTERLEAVED>(a[i], b[i], x0, x1);
        if (weight) {
            const float inv = inverse_norm<LPH>(x0, x1, p.D, p.eps);
            if (mine) {
                uint64_t w0[4], w1[4];
                spread<INTERLEAVED>(*reinterpret_cast<const uint4 *>(weight + at0),
                                    *reinterpret_cast<const uint4 *>(weight + at1), w0, w1);
                const uint64_t inv2 = f2(inv, inv);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x0[e] = mul2(mul2(x0[e], inv2), w0[e]);
                    x1[e] = mul2(mul2(x1[e], inv2), w1[e]);
                }
            }
        }
        if (h < 0) continue;
        uint4 ya, yb;
        if (kind[i] == 1 && p.k_plain) {
            gather<INTERLEAVED>(x0, x1, ya, yb);
            put(p.k_plain + t * p.k_plain_stride, h, ya, yb);
        }
        if (pos != 0) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint64_t y0, y1;
                rotate2(x0[e], x1[e], cs[2 * e], cs[2 * e + 1], y0, y1);
                x0[e] = y0;
                x1[e] = y1;
            }
        }
        gather<INTERLEAVED>(x0, x1, ya, yb);
        if (kind[i] == 0) {
            put(p.q_out + t * p.q_out_stride, h, ya, yb);
            continue;
        }
        if (p.k_out) put(p.k_out + t * p.k_out_stride, h, ya, yb);
        if (page) put(page, h, ya, yb);
    }
}

template <int LPH, bool INTERLEAVED>
cudaError_t run_norm_rope(NormRopeParams p, cudaStream_t s)
{
    constexpr int kHeads = 32 / LPH;
    p.units_q = p.q ? (p.Hq + kHeads - 1) / kHeads : 0;
    p.units_k = (p.H + kHeads - 1) / kHeads;
    p.units = p.units_q + p.units_k + (p.v ? p.units_k : 0);
    const int most = p.T * p.units > 8 * (int64_t)kPlanSms * kNormWarps ? 4 : 1;
    p.warps = (p.units + most - 1) / most;
    const int64_t blocks = (p.T * p.warps + kNormWarps - 1) / kNormWarps;
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    if (most == 4)
        return launch_chained(norm_rope_kernel<LPH, INTERLEAVED, 4>, dim3((unsigned)blocks), kNormWarps * 32, 0, s, p);
    return launch_chained(norm_rope_kernel<LPH, INTERLEAVED, 1>, dim3((unsigned)blocks), kNormWarps * 32, 0, s, p);
}

template <bool INTERLEAVED>
cudaError_t run_norm_rope(const NormRopeParams &p, cudaStream_t s)
{
    if (p.D <= 16) return run_norm_rope<1, INTERLEAVED>(p, s);
    if (p.D <= 32) return run_norm_rope<2, INTERLEAVED>(p, s);
    if (p.D <= 64) return run_norm_rope<4, INTERLEAVED>(p, s);
    if (p.D <= 128) return run_norm_rope<8, INTERLEAVED>(p, s);
    return run_norm_rope<16, INTERLEAVED>(p, s);
}

bool bad_rows(const void *ptr, int64_t stride, int64_t wide)
{
    return reinterpret_cast<uintptr_t>(ptr) % 16 || stride % 8 || stride < wide;
}

}  // namespace

}  // namespace kvi

using namespace kvi;

extern "C" kvi_status kvi_norm_rope(const kvi_attention *a, const kvi_rope *rope, int32_t max_position, int64_t T,
                                    const int32_t *d_positions, const void *d_q, int64_t q_row_stride, const void *d_k,
                                    int64_t k_row_stride, const void *d_q_weight, const void *d_k_weight, float eps,
                                    void *d_q_out, int64_t q_out_row_stride, void *d_k_out, int64_t k_out_row_stride,
                                    void *d_k_plain, int64_t k_plain_row_stride, const void *d_v, int64_t v_row_stride,
                                    const kvi_paged_cache *cache, int32_t layer, const int64_t *d_slots,
                                    int32_t *d_status, kvi_stream_t stream)
{
    kvi_status st = check_attention(a);
    if (st != KVI_OK) return st;
    if (T < 0 || T > (1 << 28)) return arg_error("T=%lld outside [0, 2^28]", (long long)T);
    const int64_t wq = (int64_t)a->q_heads * a->head_dim, wk = (int64_t)a->kv_heads * a->head_dim;
    if (unusable(d_status, 4) || (T && (unusable(d_positions, 4) || !d_k)))
        return arg_error("a required pointer (positions, k, status) is NULL, or one is misaligned");
    if (T && !d_q != !d_q_out) return arg_error("q and q_out go together");
    if (T && !d_k_out && !d_k_plain && !cache) return arg_error("k goes nowhere: no k_out, k_plain or cache");
    if (cache) {
        const int32_t none = 0;
        st = check_pages(cache, layer, 1, 1, &none);
        if (st != KVI_OK) return st;
        if (T && (!d_v || unusable(d_slots, 8))) return arg_error("a cache needs v and slots (8-byte aligned)");
    } else if (d_v || d_slots) {
        return arg_error("v and slots need a cache");
    }
    if ((d_q && (bad_rows(d_q, q_row_stride, wq) || bad_rows(d_q_out, q_out_row_stride, wq))) ||
        (d_k && bad_rows(d_k, k_row_stride, wk)) || (d_v && bad_rows(d_v, v_row_stride, wk)) ||
        (d_k_out && bad_rows(d_k_out, k_out_row_stride, wk)) ||
        (d_k_plain && bad_rows(d_k_plain, k_plain_row_stride, wk)))
        return arg_error("rows must be 16-byte aligned, with strides of at least heads * head_dim elements");
    if (reinterpret_cast<uintptr_t>(d_q_weight) % 16 || reinterpret_cast<uintptr_t>(d_k_weight) % 16)
        return arg_error("weights must be 16-byte aligned");
    if ((d_q_weight || d_k_weight) && !(eps >= 1e-12f && eps <= 1.f)) return arg_error("eps must be in [1e-12, 1]");
    if (T && d_k_plain && d_k_plain == d_k_out) return arg_error("k_plain and k_out are one buffer");
    const float4 *table;
    int32_t positions;
    st = rope_table(rope, a->head_dim, max_position, stream, &table, &positions);
    if (st != KVI_OK || T == 0) return st;
    NormRopeParams p{};
    p.q = static_cast<const __nv_bfloat16 *>(d_q);
    p.q_stride = q_row_stride;
    p.k = static_cast<const __nv_bfloat16 *>(d_k);
    p.k_stride = k_row_stride;
    p.v = static_cast<const __nv_bfloat16 *>(d_v);
    p.v_stride = v_row_stride;
    p.wq = static_cast<const __nv_bfloat16 *>(d_q_weight);
    p.wk = static_cast<const __nv_bfloat16 *>(d_k_weight);
    p.eps = eps;
    p.q_out = static_cast<__nv_bfloat16 *>(d_q_out);
    p.q_out_stride = q_out_row_stride;
    p.k_out = static_cast<__nv_bfloat16 *>(d_k_out);
    p.k_out_stride = k_out_row_stride;
    p.k_plain = static_cast<__nv_bfloat16 *>(d_k_plain);
    p.k_plain_stride = k_plain_row_stride;
    if (cache) {
        p.pool = static_cast<__nv_bfloat16 *>(cache->layer_base[layer]);
        p.n_slots = (int64_t)cache->num_blocks * cache->block_size;
        p.plane = p.n_slots * wk;
        p.slots = d_slots;
    }
    p.positions = d_positions;
    p.max_position = std::min(max_position, positions);
    p.table = table;
    p.T = T;
    p.Hq = a->q_heads;
    p.H = a->kv_heads;
    p.D = a->head_dim;
    p.status = d_status;
    return cuda_status(rope->pairing == KVI_ROPE_PAIR_INTERLEAVED ? run_norm_rope<true>(p, stream)
                                                                  : run_norm_rope<false>(p, stream),
                       "kvi_norm_rope");
}
