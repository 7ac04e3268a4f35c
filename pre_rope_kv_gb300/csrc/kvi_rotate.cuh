// kvi_rotate.cuh -- the rotation of bf16 rows by the table's cos/sin pairs
// (Section 5.1, Chunked RoPE), shared by the kernels that inject stored keys
// and that rotate a step's own queries and keys, so that both give the same
// bits.  Its accuracy is described in kvi_inject.cu.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace kvi {
namespace {

__device__ __forceinline__ uint32_t bf16_pair(float a, float b)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);  // .x = a (low half)
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Packed float32 pairs (Blackwell .f32x2 arithmetic): two adjacent
// frequencies are rotated by one instruction.  Each op rounds each half to
// nearest, exactly as the scalar op would.
__device__ __forceinline__ uint64_t f2(float lo, float hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// bf16x2 (low half = first element) -> float32 pair
__device__ __forceinline__ uint64_t bf2_to_f2(uint32_t u)
{
    return f2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
// float32 pair -> bf16x2, round to nearest even
__device__ __forceinline__ uint32_t f2_to_bf2(uint64_t v)
{
    float lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
    return bf16_pair(lo, hi);
}

// Rotate 8 rotate-half pairs: lo holds x_i, hi holds x_{i+D/2}, for
// i = 8v .. 8v+7.  cs holds the table entries of those pairs, two pairs per
// 32 bytes: {cos_hi[i], cos_hi[i+1], cos_lo[i], cos_lo[i+1]},
// {sin_hi[i], sin_hi[i+1], sin_lo[i], sin_lo[i+1]}.  x * hi products are exact
// (8 x 16 significant bits), so y0 = x0 c - x1 s and y1 = x1 c + x0 s get one
// rounding of their main part plus a float32 tail correction.
// Rotate two pairs at once: x0 holds their first elements, x1 their second,
// c / sn the pairs' table entries.
__device__ __forceinline__ void rotate2(uint64_t x0, uint64_t x1, const float4 &c, const float4 &sn,
                                        uint64_t &y0, uint64_t &y1)
{
    const uint64_t chi = f2(c.x, c.y), clo = f2(c.z, c.w);
    const uint64_t shi = f2(sn.x, sn.y), slo = f2(sn.z, sn.w);
    y0 = add2(sub2(mul2(x0, chi), mul2(x1, shi)), sub2(mul2(x0, clo), mul2(x1, slo)));
    y1 = add2(add2(mul2(x1, chi), mul2(x0, shi)), add2(mul2(x1, clo), mul2(x0, slo)));
}

__device__ __forceinline__ void rotate8(uint4 &lo, uint4 &hi, const float4 *cs)
{
    uint32_t *pl = reinterpret_cast<uint32_t *>(&lo);
    uint32_t *ph = reinterpret_cast<uint32_t *>(&hi);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        uint64_t y0, y1;
        rotate2(bf2_to_f2(pl[w]), bf2_to_f2(ph[w]), cs[2 * w], cs[2 * w + 1], y0, y1);
        pl[w] = f2_to_bf2(y0);
        ph[w] = f2_to_bf2(y1);
    }
}

// Interleaved pairing: 16 consecutive elements a (8) then b (8) hold pairs
// (2i, 2i+1) for 8 consecutive i, one pair per 32-bit word.  The first and
// second elements of two adjacent pairs are gathered into float32 pairs,
// rotated as above and interleaved back.
__device__ __forceinline__ void rotate8_interleaved(uint4 &a, uint4 &b, const float4 *cs)
{
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const uint32_t u = w[2 * g], v = w[2 * g + 1];
        const uint64_t x0 = f2(__uint_as_float(u << 16), __uint_as_float(v << 16));
        const uint64_t x1 = f2(__uint_as_float(u & 0xffff0000u), __uint_as_float(v & 0xffff0000u));
        uint64_t y0, y1;
        rotate2(x0, x1, cs[2 * g], cs[2 * g + 1], y0, y1);
        float y0a, y0b, y1a, y1b;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(y0a), "=f"(y0b) : "l"(y0));
        asm("mov.b64 {%0, %1}, %2;" : "=f"(y1a), "=f"(y1b) : "l"(y1));
        w[2 * g] = bf16_pair(y0a, y1a);
        w[2 * g + 1] = bf16_pair(y0b, y1b);
    }
    a = make_uint4(w[0], w[1], w[2], w[3]);
    b = make_uint4(w[4], w[5], w[6], w[7]);
}

}  // namespace
}  // namespace kvi
