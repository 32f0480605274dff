// mbarrier.cuh -- shared-memory mbarriers for bulk copies, with bounded waits.
//
// A wait gives up after kWaitLimitNs of %globaltimer and says so; callers
// turn that into an error they can report instead of hanging.  A thread that
// was kept from looking (its context switched out, a debugger) is charged
// kPauseNs for the gap however long it was, so that it looks again before it
// gives up.

#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace {

#ifdef FP8Q_TEST_HOOKS  // tests make waits run out
constexpr uint64_t kWaitLimitNs = 100000000ull;
#else
constexpr uint64_t kWaitLimitNs = 1000000000ull;  // one second
#endif
constexpr uint64_t kPauseNs = 10000000ull;

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ uint64_t global_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

__device__ __forceinline__ void mbar_init(uint64_t* bar) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_addr(bar)) : "memory");
}

// Start a copy of `bytes` (a multiple of 16, both addresses 16-byte aligned)
// from global memory into shared memory; its completion flips *bar's phase.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes)
                 : "memory");
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            smem_addr(dst)),
        "l"(src), "r"(bytes), "r"(smem_addr(bar))
        : "memory");
}

// How long a wait has looked in vain: more() after each look that found nothing.
struct WaitClock {
    uint64_t last = 0, spent = 0;
    __device__ __forceinline__ bool more() {
        const uint64_t t = global_ns();
        if (last) spent += t - last < kPauseNs ? t - last : kPauseNs;
        last = t;
        return spent <= kWaitLimitNs;
    }
};

__device__ __forceinline__ bool mbar_try(uint64_t* bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return done != 0;
}

// Wait until *bar has completed the phase of the given parity; false if that
// has not happened within kWaitLimitNs.  Each thread finds out for itself:
// where a warp has to go on as one, mbar_wait_all() (tcgen05.cuh).
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity) {
    WaitClock clock;
    while (!mbar_try(bar, parity))
        if (!clock.more()) return false;
    return true;
}

}  // namespace
