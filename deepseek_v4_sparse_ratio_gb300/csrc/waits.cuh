// Waits that last as long as many blocks of work take.
#pragma once

#include "common.cuh"

namespace dsa {

// mbar_wait for a wait that spans whole units of work, whose length is the caller's sequence: the
// budget counts from the last time that `blocks`, the CTA's count of blocks begun, moved. So it
// ends when the CTA stands still for a budget (about a second), however slow its blocks are and
// however many: the count only rises, up to the run's length. (A budget for the whole wait is
// 2^31 cycles; two units of 2^24 tokens are 262,144 blocks, at 4,300 to 7,100 cycles a block 1.1
// to 1.9 times 10^9.)
static __device__ __noinline__ bool wait_moving(uint64_t *bar, uint32_t parity,
                                                volatile int *abort,
                                                const volatile uint32_t *blocks, int32_t *status) {
    const uint32_t b = smem_u32(bar);
    long long t0 = clock64();
    uint32_t seen = *blocks;
    while (!mbar_test(b, parity)) {
        if (*abort) return false;
        const uint32_t now = *blocks;
        const long long t = clock64();
        if (now != seen) {
            seen = now;
            t0 = t;
        } else if (t - t0 > kWaitBudget) {
            *abort = 1;
            report(status, DSA_ERR_TIMEOUT);
            return false;
        }
    }
    return true;
}

}  // namespace dsa
