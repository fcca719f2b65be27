// A row of the 4-bit pages: where its parts lie, and what its codes stand for.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "paged.h"

namespace dsa {

constexpr int kQ4Row = DSA_Q4_ROW_BYTES;
constexpr int kQ4Dims = kD - kRope;    // dims held in 4 bits
constexpr int kQ4Rope = 32 + kQ4Dims / 2;  // first byte of the bf16 dims
static_assert(kQ4Rope + 2 * kRope == kQ4Row, "a row's parts");

__device__ __forceinline__ float pow2(int e) {  // -126 <= e <= 127
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// What an e4m3 byte stands for (0x7F: NaN).
__device__ __forceinline__ float e4m3(uint32_t byte) {
    return __half2float(
        __half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(byte), __NV_E4M3)));
}

// E from the row's byte. 14 to 250 are written; other memory may hold any, and counts as the nearest
// of these in every reader: below 14, halves of the smallest values would be no bf16, and above 250
// the values of the largest scales no finite ones (72 u, u = 448 2^113 at most, is 2^127.98).
__device__ __forceinline__ int q4_exp(uint32_t b) {
    return min(max(static_cast<int>(b), 14), 250) - 137;
}

// A scale times the row's power of two: s 2^E.
__device__ __forceinline__ float q4_unit(uint32_t scale, uint32_t b) {
    return e4m3(scale) * pow2(q4_exp(b));
}

// Dims 2 k and 2 k + 1 of a word of eight codes, as two bf16: (n + 8) 2 + 128 = 144 + 2 n has its
// bits below those of 128, and (144 + 2 n) (u / 2) - 72 u = n u in one rounding that is none:
// n u has at most seven significant bits, 72 u = 9 u 2^3 eight, and u / 2 is 2^-133 at least.
// `half` is u / 2 and `off` -72 u, each twice.
__device__ __forceinline__ uint32_t q4_pair(uint32_t word, int k, __nv_bfloat162 half,
                                            __nv_bfloat162 off) {
    const uint32_t c = k == 0 ? word << 1 : word >> (4 * k - 1);
    const uint32_t x = (c & 0x001E001Eu) | 0x43004300u;
    const __nv_bfloat162 y =
        __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&x), half, off);
    return *reinterpret_cast<const uint32_t *>(&y);
}

}  // namespace dsa
