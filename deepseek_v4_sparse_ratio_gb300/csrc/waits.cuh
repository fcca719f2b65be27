// Waits that may last as long as many blocks of work take.
#pragma once

#include "common.cuh"

namespace dsa {

// The CTA's count of blocks begun lies this many words behind its abort flag.
constexpr int kBlocksAt = 8;

// mbar_wait for kernels whose waits may span whole units of work, as long as the caller's
// sequences: when the budget is used up it starts anew if the CTA has begun a block since the last
// time. So it ends when the CTA stands still for one budget (about a second) to two, however slow
// its blocks are and however many: the count only rises, up to the run's length. (One budget for
// the whole wait is 2^31 cycles; two units of 2^24 tokens are 262,144 blocks, at 4,300 to 7,100
// cycles a block 1.1 to 1.9 times 10^9.) Out of line: its many copies would push the roles' code
// out of the instruction caches.
static __device__ __noinline__ bool wait_moving(uint64_t *bar, uint32_t parity,
                                                volatile int *abort, int32_t *status) {
    const uint32_t b = smem_u32(bar);
    int seen = abort[kBlocksAt];
    long long t0 = clock64();
    while (!mbar_test(b, parity)) {
        if (*abort) return false;
        if (clock64() - t0 > kWaitBudget) {
            const int now = abort[kBlocksAt];
            if (now == seen) {
                *abort = 1;
                report(status, DSA_ERR_TIMEOUT);
                return false;
            }
            seen = now;
            t0 = clock64();
        }
    }
    return true;
}

}  // namespace dsa
