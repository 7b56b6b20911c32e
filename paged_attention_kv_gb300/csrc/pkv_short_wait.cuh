// The bounded waits of prompt_kernel. pkv_selftest_bounded_wait runs them too.
#pragma once

#include <cstdint>

#include "pkv_device.cuh"

namespace pkv {

// Bounded waits: after timeout_ns, or once another wait has given up, they set
// *abort and return false; the CTA reports PKV_DEV_TIMEOUT when it ends. They
// are short, since each is in the code many times and all roles share the
// instruction cache (at 108 KB of code short prompts ran a fifth slower than
// at 78 KB); and there is no call in them: values that live across a call are
// kept out of uniform registers, where the MMA instructions want them (60 to 90
// cycles an MMA instead of 15, more than the tensor core's 64), and a role's
// larger share of registers would not pass through one.
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}
__device__ __forceinline__ uint32_t timer_lo() {
    uint32_t t;
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
    return t;
}
__device__ __forceinline__ bool is_done(uint32_t bar, uint32_t parity) {  // asked by a whole warp, without waiting
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return __all_sync(0xffffffffu, done != 0);
}
// By a whole warp, which leaves it with one answer.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort,
                                          uint32_t timeout_ns = (uint32_t)kWaitTimeoutNs) {
    uint32_t t0 = 0;
#pragma unroll 1
    while (!__all_sync(0xffffffffu, try_wait(bar, parity))) {
        const uint32_t now = timer_lo();
        t0 = t0 ? t0 : now | 1;
        if (__any_sync(0xffffffffu, now - t0 + 1 > timeout_ns || *abort)) {
            *abort = 1;
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
    return warp_wait(smem_u32(bar), parity, abort);
}
// By one thread.
__device__ __forceinline__ bool lane_wait(uint64_t *bar, uint32_t parity, volatile int *abort,
                                          uint32_t timeout_ns = (uint32_t)kWaitTimeoutNs) {
    const uint32_t b = smem_u32(bar), t0 = timer_lo();
    while (!try_wait(b, parity)) {
        if (timer_lo() - t0 > timeout_ns || *abort) {
            *abort = 1;
            return false;
        }
    }
    return true;
}

}  // namespace pkv
