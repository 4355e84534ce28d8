// wait.cuh -- bounded device waits: on expiry the waiter records
// MOE_ERR_TIMEOUT in the context's status word and gives up.
#pragma once
#include "common.cuh"
#include "ptx.cuh"

namespace moeq4 {

constexpr unsigned long long kWaitNs = 2000000000ull;   // bound of every device wait (2 s)

__device__ __forceinline__ unsigned long long gtimer_ns() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

__device__ __forceinline__ void fused_fail(int* status) { atomicCAS(status, 0, MOE_ERR_TIMEOUT); }

__device__ __forceinline__ bool fused_aborted(const int* status) {
    return ld_relaxed_s32(status) != 0;
}

// Waits longer than this look at the status word in global memory (a load
// that can take microseconds under load, so ordinary waits never issue it).
constexpr unsigned long long kAbortCheckNs = 20000;

// Wait on an mbarrier phase, bounded in time; once the wait is long, gives up
// early when another thread has already recorded a failure.
__device__ __forceinline__ bool fused_wait_bar(uint64_t* bar, uint32_t parity, int* status,
                                               unsigned long long bound = kWaitNs) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = gtimer_ns();
    for (unsigned it = 1;; it++) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 31) == 0) {
            const unsigned long long el = gtimer_ns() - t0;
            if (el > bound) { fused_fail(status); return false; }
            if (el > kAbortCheckNs && fused_aborted(status)) return false;
        }
    }
}

// The same for kernels whose warps wait often beside others that work: the
// hardware suspends the thread up to a microsecond at a time, where polling would
// take issue slots from the working warps.
__device__ __forceinline__ bool mbar_try_wait_long(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, int* status, unsigned long long bound) {
    if (mbar_try_wait_long(bar, parity)) return true;
    const unsigned long long t0 = gtimer_ns();
    while (!mbar_try_wait_long(bar, parity)) {
        const unsigned long long el = gtimer_ns() - t0;
        if (el > bound) { fused_fail(status); return false; }
        if (el > kAbortCheckNs && fused_aborted(status)) return false;
    }
    return true;
}

}  // namespace moeq4
