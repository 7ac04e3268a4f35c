// Shared-memory barrier helpers with bounded waits, for the kernels that
// stage data through mbarrier-tracked copies (the inject kernel) and for the
// diagnostic that shows a wait giving up.  Every wait takes a time limit in
// nanoseconds of %globaltimer and reports whether the phase completed, so a
// caller can record KVI_ERR_TIMEOUT and return instead of hanging.
#pragma once
#include <cstdint>

#include <cuda_runtime.h>

namespace kvi {
namespace {

__device__ __forceinline__ uint32_t smem_u32(const void *p)
{
    return (uint32_t)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        "selp.u32 %0, 1, 0, p;\n"
        "}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ uint64_t global_ns()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// Wait for the phase with the given parity to complete; false after the
// time limit.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns)
{
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    for (;;) {
        if (mbar_try_wait(bar, parity)) return true;
        if (global_ns() - t0 > limit_ns) return false;
    }
}

// mbar_wait for waits that a kernel's pace depends on: the clock, whose
// reading takes longer than a try, is read once in 32 tries.
__device__ __forceinline__ bool mbar_wait_brisk(uint32_t bar, uint32_t parity, uint64_t limit_ns)
{
    uint64_t t0 = 0;
    for (uint32_t n = 0;; ++n) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((n & 31u) == 31u) {
            const uint64_t t = global_ns();
            if (t0 == 0) t0 = t;
            if (t - t0 > limit_ns) return false;
        }
    }
}

}  // namespace
}  // namespace kvi
