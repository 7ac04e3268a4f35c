// kvi_norm_rope.cu -- a step's own queries and keys: normalised per head,
// rotated to their positions (Section 5.1's rotation, under the conventions of
// kvi_rope) and, with the values, put into the paged cache (Section 3.4's
// scatter), in one pass.
//
//   y = x / sqrt(mean x^2 + eps) * w            (or y = x, without a weight)
//   out_i = y_i cos(p w_i) - y_j sin(p w_i),  out_j = y_j cos + y_i sin
//
// A warp takes a token's heads 32 / LPH at a time (a unit): LPH lanes hold a head,
// 16 channels each (both elements of 8 pairs), so that the norm is a few shuffles
// and the rotation none.  A lane's 8 coefficient pairs serve all heads that its
// warp takes.  Squares are summed in float32, and y stays float32 until the one
// rounding of each result; the rotation is that of the injected keys, so without
// a weight a key gets the same bits as kvi_inject_paged gives it.
//
// What bounds it: HBM.  8192 rows of 32 + 8 + 8 heads of 128, to q, the pages and
// plain keys, 40 us, 5.3 TB/s, 78 % of a copy: a warp stays with a part of the
// rows, whose weights it keeps, and bulk copies fetch its next two meanwhile.  (A
// warp per 4 units that loads, computes and ends, however many of them an SM
// holds: 50 us and more; with a lane's table entries loaded directly, 52 us.)
// Few rows are a launch and a chain of latencies: 64 rows 2.3 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "kvi_attn.cuh"
#include "kvi_rotate.cuh"
#include "kvi_sync.cuh"

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
    int32_t parts;    // of a row, in the streaming form
    float eps;
    int32_t *status;
};

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t neg2(uint64_t a) { return a ^ 0x8000000080000000ull; }
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
            const uint64_t a = f == 1.f ? x0[i] : mul2(x0[i], ff), b = f == 1.f ? x1[i] : mul2(x1[i], ff);
            s = fma2(b, b, fma2(a, a, s));
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

// What a lane is to do with a unit (32 / LPH heads of one kind) of a row.
enum : int { kQ = 0, kK = 1, kV = 2, kNone = 3 };
template <int LPH>
__device__ __forceinline__ int unit_kind(const NormRopeParams &p, int u, int &head0)
{
    const int kind = u >= p.units ? kNone : u < p.units_q ? kQ : u < p.units_q + p.units_k ? kK : kV;
    head0 = (u - (kind == kQ ? 0 : kind == kK ? p.units_q : p.units_q + p.units_k)) * (32 / LPH);
    return kind;
}
__device__ __forceinline__ const __nv_bfloat16 *unit_rows(const NormRopeParams &p, int kind, int64_t t)
{
    return kind == kQ ? p.q + t * p.q_stride : kind == kK ? p.k + t * p.k_stride : p.v + t * p.v_stride;
}

// A lane's 16 channels of a row's heads, with the row's coefficients.  NORMED:
// both weights are there, and are multiplied with them.
template <int LPH, bool INTERLEAVED, bool NORMED>
struct Lane {
    const NormRopeParams &p;
    int at0, at1;  // its two pieces of 8 channels
    bool mine;     // (heads of fewer than LPH lanes)
    int64_t t;
    int32_t pos;
    __nv_bfloat16 *page;
    float4 cs[8];
    uint64_t wc0[4], wc1[4], ws0[4], ws1[4];  // weights times cosines; times sines, the second elements' minus

    __device__ __forceinline__ Lane(const NormRopeParams &params) : p(params)
    {
        const int c = (threadIdx.x & 31) % LPH;
        at0 = INTERLEAVED ? 16 * c : 8 * c;
        at1 = INTERLEAVED ? at0 + 8 : p.D / 2 + at0;
        mine = 16 * c < p.D;
    }
    // The row, and its entries of the table, of which a lane wants 8 in a row (128
    // bytes): they come in coalesced and go through shared memory, entry e of lane
    // c at e * kPitch + c.
    static constexpr int kPitch = LPH + 1, kLoads = (8 * LPH + 31) / 32;
    __device__ __forceinline__ void ask_table(int32_t position, float4 (&ahead)[kLoads]) const
    {
        const float4 *row = p.table + (int64_t)position * (p.D / 2);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int at = i * 32 + (int)(threadIdx.x & 31);
            ahead[i] = at < p.D / 2 ? __ldg(row + at) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    __device__ __forceinline__ void take_row(int64_t token, int32_t position, int64_t slot, const float4 (&ahead)[kLoads],
                                             float4 *stage)
    {
        const int lane = threadIdx.x & 31;
        t = token;
        pos = position;
        page = slot < 0 ? nullptr : p.pool + slot * ((int64_t)p.H * p.D);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int at = i * 32 + lane;
            if (at < 8 * LPH) stage[(at & 7) * kPitch + (at >> 3)] = ahead[i];
        }
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; ++e) cs[e] = stage[e * kPitch + lane % LPH];
    }
    __device__ __forceinline__ void put(__nv_bfloat16 *dst, int head, const uint4 &x, const uint4 &y) const
    {
        dst += (int64_t)head * p.D;
        *reinterpret_cast<uint4 *>(dst + at0) = x;
        *reinterpret_cast<uint4 *>(dst + at1) = y;
    }
    __device__ __forceinline__ void weights(int kind, uint64_t (&w0)[4], uint64_t (&w1)[4]) const
    {
        const __nv_bfloat16 *w = kind == kQ ? p.wq : p.wk;
        const uint4 zero = make_uint4(0, 0, 0, 0);
        spread<INTERLEAVED>(mine ? *reinterpret_cast<const uint4 *>(w + at0) : zero,
                            mine ? *reinterpret_cast<const uint4 *>(w + at1) : zero, w0, w1);
    }
    __device__ __forceinline__ void set_kind(int kind)
    {
        if (!NORMED) return;
        weights(kind, wc0, wc1);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint64_t cosine = add2(f2(cs[2 * e].x, cs[2 * e].y), f2(cs[2 * e].z, cs[2 * e].w));
            const uint64_t sine = add2(f2(cs[2 * e + 1].x, cs[2 * e + 1].y), f2(cs[2 * e + 1].z, cs[2 * e + 1].w));
            ws0[e] = mul2(wc0[e], sine);
            ws1[e] = neg2(mul2(wc1[e], sine));
            wc0[e] = mul2(wc0[e], cosine);
            wc1[e] = mul2(wc1[e], cosine);
        }
    }
    // A head of q, k or v (a, b: its channels; head < 0: none here).  Every lane of
    // the warp comes along.
    __device__ __forceinline__ void finish(int kind, int head, const uint4 &a, const uint4 &b) const
    {
        if (kind == kV) {
            if (head >= 0 && page) put(page + p.plane, head, a, b);
            return;
        }
        uint64_t x0[4], x1[4], y0[4], y1[4];
        uint4 ya, yb;
        spread<INTERLEAVED>(a, b, x0, x1);
        const bool weighted = NORMED || (kind == kQ ? p.wq : p.wk) != nullptr;
        if (weighted) {
            const float inv = inverse_norm<LPH>(x0, x1, p.D, p.eps);
            const uint64_t inv2 = f2(inv, inv);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x0[e] = mul2(x0[e], inv2);
                x1[e] = mul2(x1[e], inv2);
            }
        }
        if (head < 0) return;
        if (weighted && (!NORMED || (kind == kK && p.k_plain))) {
            weights(kind, y0, y1);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                y0[e] = mul2(x0[e], y0[e]);
                y1[e] = mul2(x1[e], y1[e]);
                if (!NORMED) {
                    x0[e] = y0[e];
                    x1[e] = y1[e];
                }
            }
        }
        if (kind == kK && p.k_plain) {
            if (NORMED)
                gather<INTERLEAVED>(y0, y1, ya, yb);
            else
                gather<INTERLEAVED>(x0, x1, ya, yb);
            put(p.k_plain + t * p.k_plain_stride, head, ya, yb);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (NORMED) {
                y0[e] = fma2(x1[e], ws1[e], mul2(x0[e], wc0[e]));
                y1[e] = fma2(x1[e], wc1[e], mul2(x0[e], ws0[e]));
            } else if (pos != 0) {
                rotate2(x0[e], x1[e], cs[2 * e], cs[2 * e + 1], y0[e], y1[e]);
            } else {  // (its bits, as an injected key's)
                y0[e] = x0[e];
                y1[e] = x1[e];
            }
        }
        gather<INTERLEAVED>(y0, y1, ya, yb);
        if (kind == kQ) {
            put(p.q_out + t * p.q_out_stride, head, ya, yb);
            return;
        }
        if (p.k_out) put(p.k_out + t * p.k_out_stride, head, ya, yb);
        if (page) put(page, head, ya, yb);
    }
};

// Few rows: a warp for each unit.
template <int LPH, bool INTERLEAVED, bool NORMED>
__global__ void __launch_bounds__(kNormWarps * 32) norm_rope_kernel(const __grid_constant__ NormRopeParams p)
{
    using L = Lane<LPH, INTERLEAVED, NORMED>;
    __shared__ float4 s_table[kNormWarps][8 * L::kPitch];
    const uint32_t w = blockIdx.x * kNormWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int64_t t = w / (uint32_t)p.units;
    pdl_wait();
    pdl_launch_dependents();
    if (t >= p.T) return;
    L l(p);
    int head0;
    const int kind = unit_kind<LPH>(p, (int)(w - (uint32_t)t * (uint32_t)p.units), head0);
    const int32_t pos = p.positions[t];
    int64_t slot = p.slots ? p.slots[t] : -1;
    int head = head0 + (int)lane / LPH;
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    if (l.mine && head < (kind == kQ ? p.Hq : p.H)) {
        const __nv_bfloat16 *src = unit_rows(p, kind, t) + (int64_t)head * p.D;
        a = *reinterpret_cast<const uint4 *>(src + l.at0);
        b = *reinterpret_cast<const uint4 *>(src + l.at1);
    } else {
        head = -1;
    }
    if (pos < 0 || pos >= p.max_position) {
        if (lane == 0) record_status(p.status, KVI_ERR_OUT_OF_RANGE);
        return;
    }
    if (slot >= p.n_slots) {
        if (lane == 0) record_status(p.status, KVI_ERR_OUT_OF_RANGE);
        slot = -1;
    }
    float4 entries[L::kLoads];
    l.ask_table(pos, entries);
    l.take_row(t, pos, slot, entries, s_table[threadIdx.x >> 5]);
    if (kind != kV) l.set_kind(kind);
    l.finish(kind, head, a, b);
}

// Many rows, head sizes of 64, 128 and 256: a warp stays with its part of a row
// (four units of q, or two of k with the two of v beside them) and goes from row to
// row; bulk copies bring the next ones' into a ring of its own meanwhile.
constexpr int kPartUnits = 4, kRowStages = 3, kRowBlocks = 3;
constexpr int kUnitBytes = 1024;  // 32 lanes of 16 channels
constexpr uint64_t kRowWaitNs = 1000000000ull;

template <int D>
struct StreamSmem {
    uint8_t rows[kNormWarps][kRowStages][kPartUnits * kUnitBytes];
    float4 table[kNormWarps][8 * (D / 16 + 1)];
    uint64_t full[kNormWarps][kRowStages];
};

template <int D, bool INTERLEAVED, bool NORMED>
__global__ void __launch_bounds__(kNormWarps * 32, kRowBlocks) norm_rope_stream(const __grid_constant__ NormRopeParams p)
{
    constexpr int LPH = D / 16, kHeads = 32 / LPH, kLoads = (8 * LPH + 31) / 32, kPitch = LPH + 1;
    extern __shared__ __align__(128) uint8_t smem[];
    StreamSmem<D> &sm = *reinterpret_cast<StreamSmem<D> *>(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane % LPH, sub = lane / LPH;
    const int at0 = sub * D + (INTERLEAVED ? 16 * c : 8 * c), at1 = at0 + (INTERLEAVED ? 8 : D / 2);  // in a unit
    const uint32_t w = blockIdx.x * kNormWarps + warp;
    const int64_t step = gridDim.x * kNormWarps / (uint32_t)p.parts;
    const int64_t t0 = w / (uint32_t)p.parts;
    int part = (int)(w - (uint32_t)t0 * (uint32_t)p.parts);
    const uint32_t full0 = smem_u32(&sm.full[warp][0]), rows0 = smem_u32(&sm.rows[warp][0][0]);
    if (lane < kRowStages) mbar_init(full0 + 8 * lane, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    pdl_wait();
    pdl_launch_dependents();
    if (t0 >= step) return;  // (warps past the last whole row of parts)
    // ---- this warp's part, and this lane's copies: q, or k and (lane 1) v
    const int parts_q = (p.units_q + kPartUnits - 1) / kPartUnits;
    const bool is_q = part < parts_q;
    if (!is_q) part -= parts_q;
    constexpr int kHalfPart = kPartUnits / 2 * kHeads;  // heads of k, and of v
    const int head0 = part * (is_q ? kPartUnits * kHeads : kHalfPart);
    const int heads = min(is_q ? kPartUnits * kHeads : kHalfPart, (is_q ? p.Hq : p.H) - head0);
    const __nv_bfloat16 *src = nullptr;
    int64_t src_step = 0;
    if (lane == 0) {
        src = is_q ? p.q : p.k;
        src_step = is_q ? p.q_stride : p.k_stride;
    } else if (lane == 1 && !is_q && p.v) {
        src = p.v;
        src_step = p.v_stride;
    }
    const uint32_t bytes = heads * D * 2, all = is_q || !p.v ? bytes : 2 * bytes;
    const bool copies = src != nullptr;
    src += t0 * src_step + (int64_t)head0 * D;
    src_step *= step;
    auto copy = [&](int stage) {
        if (lane == 0) mbar_expect_tx(full0 + 8 * stage, all);
        __syncwarp();
        if (copies) {
            asm volatile(
                "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                    rows0 + (stage * kPartUnits + lane * (kPartUnits / 2)) * kUnitBytes),
                "l"(src), "r"(bytes), "r"(full0 + 8 * stage)
                : "memory");
            src += src_step;
        }
    };
    int64_t asked = t0;  // next row to copy
    for (int s = 0; s < kRowStages - 1; ++s, asked += step)
        if (asked < p.T) copy(s);
    // ---- weights (in float32), outputs
    const __nv_bfloat16 *weight = is_q ? p.wq : p.wk;
    uint64_t w0[4], w1[4];
    if (NORMED || weight)
        spread<INTERLEAVED>(*reinterpret_cast<const uint4 *>(weight + at0 - sub * D),
                            *reinterpret_cast<const uint4 *>(weight + at1 - sub * D), w0, w1);
    const int64_t out0 = (int64_t)head0 * D, own = (int64_t)p.H * D;
    auto position = [&](int64_t t) { return t < p.T ? p.positions[t] : -1; };
    auto slot_of = [&](int64_t t) { return !is_q && p.slots && t < p.T ? p.slots[t] : (int64_t)-1; };
    auto known = [&](int32_t pos) { return pos >= 0 && pos < p.max_position; };
    float4 entries[kLoads];
    auto ask_table = [&](int32_t pos) {
        const float4 *row = p.table + (int64_t)(known(pos) ? pos : 0) * (D / 2);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) entries[i] = __ldg(row + i * 32 + lane);
    };
    int32_t pos = position(t0), next_pos = position(t0 + step);
    int64_t slot = slot_of(t0);
    ask_table(pos);
    int stage = 0, ahead_stage = kRowStages - 1;
    uint32_t phase = 0;
    bool ok = true;
    for (int64_t t = t0; t < p.T; t += step) {
        if (asked < p.T) copy(ahead_stage);
        asked += step;
        ahead_stage = ahead_stage + 1 == kRowStages ? 0 : ahead_stage + 1;
        if (slot >= p.n_slots) {
            if (lane == 0) record_status(p.status, KVI_ERR_OUT_OF_RANGE);
            slot = -1;
        }
        const int32_t here = pos;
        const int64_t to = slot;
        if (!known(here) && lane == 0) record_status(p.status, KVI_ERR_OUT_OF_RANGE);
        // A lane wants 8 entries of the table in a row, 128 bytes: they came in
        // coalesced and go through shared memory.
        float4 cs[8];                                   // as they are, or (NORMED)
        uint64_t wc0[4], wc1[4], ws0[4], ws1[4];        // weights times cosines; times sines, the second elements' minus
        float4 *const table = sm.table[warp];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int at = i * 32 + lane, e = at & 7, of = at >> 3;
            if (NORMED)
                reinterpret_cast<float2 *>(table)[2 * ((e >> 1) * kPitch + of) + (e & 1)] =
                    make_float2(entries[i].x + entries[i].z, entries[i].y + entries[i].w);
            else
                table[e * kPitch + of] = entries[i];
        }
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (NORMED) {
                const float4 v = table[e * kPitch + c];
                const uint64_t cosine = f2(v.x, v.y), sine = f2(v.z, v.w);
                wc0[e] = mul2(w0[e], cosine);
                wc1[e] = mul2(w1[e], cosine);
                ws0[e] = mul2(w0[e], sine);
                ws1[e] = neg2(mul2(w1[e], sine));
            } else {
                cs[2 * e] = table[2 * e * kPitch + c];
                cs[2 * e + 1] = table[(2 * e + 1) * kPitch + c];
            }
        }
        pos = next_pos;
        next_pos = position(t + 2 * step);
        slot = slot_of(t + step);
        ask_table(pos);
        ok = __all_sync(0xffffffffu, mbar_wait_brisk(full0 + 8 * stage, phase, kRowWaitNs));
        if (!ok) break;
        const __nv_bfloat16 *rows = reinterpret_cast<const __nv_bfloat16 *>(sm.rows[warp][stage]);
        if (known(here)) {
            __nv_bfloat16 *const page = to < 0 ? nullptr : p.pool + to * own + out0;
            __nv_bfloat16 *const out = is_q ? p.q_out + t * p.q_out_stride + out0
                                            : p.k_out ? p.k_out + t * p.k_out_stride + out0 : nullptr;
            __nv_bfloat16 *const plain = is_q || !p.k_plain ? nullptr : p.k_plain + t * p.k_plain_stride + out0;
#pragma unroll
            for (int i = 0; i < kPartUnits; ++i) {
                if (!is_q && i >= kPartUnits / 2) {
                    const int u = i - kPartUnits / 2;
                    if (page && u * kHeads + sub < heads) {
                        __nv_bfloat16 *dst = page + p.plane + u * kHeads * D;
                        *reinterpret_cast<uint4 *>(dst + at0) = *reinterpret_cast<const uint4 *>(rows + i * kHeads * D + at0);
                        *reinterpret_cast<uint4 *>(dst + at1) = *reinterpret_cast<const uint4 *>(rows + i * kHeads * D + at1);
                    }
                    continue;
                }
                if (i * kHeads >= heads) continue;
                const bool real = i * kHeads + sub < heads;
                uint4 a = make_uint4(0, 0, 0, 0), b = a;
                if (real) {
                    a = *reinterpret_cast<const uint4 *>(rows + i * kHeads * D + at0);
                    b = *reinterpret_cast<const uint4 *>(rows + i * kHeads * D + at1);
                }
                uint64_t x0[4], x1[4], y0[4], y1[4];
                spread<INTERLEAVED>(a, b, x0, x1);
                const bool weighted = NORMED || weight;
                if (weighted) {
                    const float inv = inverse_norm<LPH>(x0, x1, D, p.eps);
                    const uint64_t inv2 = f2(inv, inv);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x0[e] = mul2(x0[e], inv2);
                        x1[e] = mul2(x1[e], inv2);
                        if (!NORMED) {
                            x0[e] = mul2(x0[e], w0[e]);
                            x1[e] = mul2(x1[e], w1[e]);
                        }
                    }
                }
                auto put = [&](__nv_bfloat16 *dst) {
                    *reinterpret_cast<uint4 *>(dst + i * kHeads * D + at0) = a;
                    *reinterpret_cast<uint4 *>(dst + i * kHeads * D + at1) = b;
                };
                if (plain && real) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        y0[e] = NORMED ? mul2(x0[e], w0[e]) : x0[e];
                        y1[e] = NORMED ? mul2(x1[e], w1[e]) : x1[e];
                    }
                    gather<INTERLEAVED>(y0, y1, a, b);
                    put(plain);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (NORMED) {
                        y0[e] = fma2(x1[e], ws1[e], mul2(x0[e], wc0[e]));
                        y1[e] = fma2(x1[e], wc1[e], mul2(x0[e], ws0[e]));
                    } else if (here != 0) {
                        rotate2(x0[e], x1[e], cs[2 * e], cs[2 * e + 1], y0[e], y1[e]);
                    } else {  // (its bits, as an injected key's)
                        y0[e] = x0[e];
                        y1[e] = x1[e];
                    }
                }
                gather<INTERLEAVED>(y0, y1, a, b);
                if (out && real) put(out);
                if (page && real) put(page);
            }
        }
        // (read by all, and only then written to by the copies asked for next)
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        stage = stage + 1 == kRowStages ? 0 : stage + 1;
        if (stage == 0) phase ^= 1u;
    }
    if (!ok) {
        if (lane == 0) record_status(p.status, KVI_ERR_TIMEOUT);
        // no copy may still be writing when the block ends
        for (int s = 0; s < kRowStages; ++s)
            (void)mbar_wait_brisk(full0 + 8 * s, s >= stage ? phase : phase ^ 1u, kRowWaitNs);
        __syncwarp();
    }
}

template <int LPH, bool INTERLEAVED, bool NORMED>
cudaError_t run_norm_rope_as(NormRopeParams p, cudaStream_t s)
{
    if constexpr (LPH >= 4) {
        constexpr int D = 16 * LPH;
        p.parts = (p.units_q + kPartUnits - 1) / kPartUnits + (p.units_k + kPartUnits / 2 - 1) / (kPartUnits / 2);
        // A warp a unit is as fast up to a few warps an SM's scheduler (us, that and
        // staying warps; 12 units a row: 256 rows 3.3, 3.5, 512 rows 6.0, 4.9; 2 units a
        // row: 2048 rows 2.5, 4.3).
        if (p.D == D && p.T * p.units > 30 * (int64_t)kPlanSms) {
            constexpr int bytes = (int)sizeof(StreamSmem<D>);
            const cudaError_t e = smem_opt_in(norm_rope_stream<D, INTERLEAVED, NORMED>, bytes);
            if (e != cudaSuccess) return e;
            // as many blocks as find room at once (and a warp for each part at least)
            const int blocks = std::max(kPlanSms * kRowBlocks, (p.parts + kNormWarps - 1) / kNormWarps);
            return launch_chained(norm_rope_stream<D, INTERLEAVED, NORMED>, dim3((unsigned)blocks), kNormWarps * 32, bytes, s, p);
        }
    }
    const int64_t blocks = (p.T * p.units + kNormWarps - 1) / kNormWarps;
    if (blocks * kNormWarps > 0x7fffffff) return cudaErrorInvalidConfiguration;
    return launch_chained(norm_rope_kernel<LPH, INTERLEAVED, NORMED>, dim3((unsigned)blocks), kNormWarps * 32, 0, s, p);
}

template <int LPH, bool INTERLEAVED>
cudaError_t run_norm_rope(NormRopeParams p, cudaStream_t s)
{
    constexpr int kHeads = 32 / LPH;
    p.units_q = p.q ? (p.Hq + kHeads - 1) / kHeads : 0;
    p.units_k = (p.H + kHeads - 1) / kHeads;
    p.units = p.units_q + p.units_k + (p.v ? p.units_k : 0);
    return (p.wq || !p.q) && p.wk ? run_norm_rope_as<LPH, INTERLEAVED, true>(p, s)
                                  : run_norm_rope_as<LPH, INTERLEAVED, false>(p, s);
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
