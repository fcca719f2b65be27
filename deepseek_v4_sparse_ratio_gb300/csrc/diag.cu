// Self-check of the bounded-wait error path. Every kernel of the library waits
// on mbarriers through mbar_wait, which gives up after about a second, records
// DSA_ERR_TIMEOUT in the caller's status word and lets the kernel return. This
// entry point runs that same wait on a barrier that either receives its one
// arrival or receives none, or the wait whose budget starts anew with every block
// of work on a barrier whose arrival takes longer than one budget, so a caller can see the error reach the host with
// the context still usable -- without any fault, trap or endless loop.
#include "waits.cuh"

namespace dsa {

__global__ void __launch_bounds__(64) wait_selftest_kernel(int32_t arrive, int32_t *status) {
    __shared__ __align__(8) uint64_t bar;
    __shared__ int words[1 + kBlocksAt];  // the abort flag, and the count of blocks
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        words[0] = words[kBlocksAt] = 0;
        fence_barrier_init();
    }
    __syncthreads();
    if (arrive == 2 || arrive == 3) {
        if (threadIdx.x == 0) {
            wait_moving(&bar, 0, words, status);
        } else if (threadIdx.x == 32) {
            // six steps of a quarter of a budget each: moving ones, or one count for all
            volatile int *count = words + kBlocksAt;
            for (int k = 0; k < 6; ++k) {
                const long long t0 = clock64();
                while (clock64() - t0 < kWaitBudget / 4) {
                }
                if (arrive == 2) *count = k + 1;
            }
            mbar_arrive(&bar);
        }
    } else if (threadIdx.x == 0) {
        if (arrive) mbar_arrive(&bar);
        mbar_wait(&bar, 0, words, status);
    }
}

}  // namespace dsa

extern "C" int dsa_bounded_wait_selftest(int32_t arrive, int32_t *dev_status, void *stream) {
    if (!dev_status) return DSA_ERR_ARG;
    dsa::wait_selftest_kernel<<<1, 64, 0, static_cast<cudaStream_t>(stream)>>>(arrive, dev_status);
    return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}
