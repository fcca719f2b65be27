// dsa_paged_q4_append and dsa_paged_q4_read: KV rows of a ragged batch into pages of 4-bit rows,
// and back.
//
// A row of 512 bf16 becomes 384 bytes (the header has the layout): 448 whole numbers n of -7 .. 7,
// a scale s in e4m3 for each 16, a power of two 2^E for the row, x ~ n s 2^E; and the 64 rotated
// dims in bf16. Both calls take one warp per row, as the bf16 append does (two or four rows a warp,
// and blocks of 4 or 16 warps, were equal or slower). Measured as a call among others, and as one
// from a cold L2 with the 2 us of the events around it:
//   write 56,436 rows   20.0, 25.2 us (their 1,408 bytes a row need 11.9): bound by the instructions,
//                       about 350 a row, three issued a cycle
//   read 56,436 rows    14.1, 19.1 us of 11.9
//   read 135,011 rows   35.2, 37.5 us of 28.4: 0.8 of the copy rate
// (the first figures have the pages in L2, 22 and 52 MB). Up to a few thousand rows the launch counts.
#include <math.h>

#include "common.cuh"
#include "paged_walk.cuh"
#include "q4.h"

namespace dsa {

namespace {

using paged::add_pair;
using paged::fma_pair;
using paged::pair_of;

constexpr int kQ4Warps = 8;
constexpr uint32_t kQ4Limit = (124u + 127u) << 23;  // the bits of 2^124
constexpr int kQ4LeastExp = -113;

// The row of the pages that holds position p of sequence s; null (and a report) for a bad entry.
__device__ __forceinline__ uint8_t *row_of(const PagedBatch &b, uint8_t *pages, int s, int32_t p,
                                           int lane, int32_t *status) {
    const int32_t page = __ldg(b.page_table + int64_t{s} * b.max_pages + (p >> b.page_shift));
    if (page < 0 || page >= b.n_pages) {
        if (lane == 0) report(status, DSA_ERR_BOUNDS);
        return nullptr;
    }
    return pages + page * b.page_stride + int64_t{p & ((1 << b.page_shift) - 1)} * kQ4Row;
}

__device__ __forceinline__ void report_bad(const PagedBatch &b, int32_t *status) {
    if (blockIdx.x != 0) return;
    for (int s = threadIdx.x; s < b.n_seqs; s += blockDim.x) {
        bool bad;
        paged_seq(b, s, bad);
        if (bad) report(status, DSA_ERR_BOUNDS);
    }
}

// The sequence and position of row r; false where it belongs to none.
__device__ __forceinline__ bool find_row(const PagedBatch &b, int64_t r, int lane, int &s,
                                         int32_t &p) {
    s = find_seq(b, r, lane);
    bool bad;
    PagedSeq q = paged_seq(b, s, bad);
    if (!holds(q, r)) {
        s = find_seq_any(b, r, lane);
        if (s < 0) return false;
        q = paged_seq(b, s, bad);
    }
    p = q.len - q.n + static_cast<int32_t>(r - q.row0);
    return true;
}

// x / s rounded to a whole number of -7 .. 7, ties to even, plus 8, from x and 1 / s (0 for 8 or
// where the group holds what is not finite). x has eight significant bits and s four, so a quotient
// of 0.4 or more that is no tie is 2^-10.9 or more from one; the product with the rounded 1 / s is
// 2^-19 off at most. Rounded to a multiple of 2^-11 first (by adding 6,144, whose last bit that
// is), ties are ties and nothing else is.
constexpr float kSnap = 6144.0f;
constexpr float kWhole = 12582912.0f + 8.0f;   // 1.5 2^23 + 8: the last bit is 1
__device__ __forceinline__ uint32_t whole_plus8(float x, float per, bool finite) {
    const float t = __fadd_rn(fmaf(x, per, kSnap), -kSnap);
    const float n = fminf(fmaxf(finite ? t : 0.0f, -7.0f), 7.0f);
    return __float_as_uint(__fadd_rn(n, kWhole)) & 15u;
}

// The same for four words of two elements each, without the bounds, in a code word's order.
// Two elements an instruction; a sum in base 16 of the bits of n + kWhole, which are n + 8 above
// those of kWhole - 8.
__device__ __forceinline__ uint32_t eight_plain(const uint32_t *w, float per) {
    // (the last addition takes kSnap off as well: kWhole - kSnap is whole, nothing rounds twice)
    const uint64_t p2 = pair_of(per), snap = pair_of(kSnap), whole = pair_of(kWhole - kSnap);
    uint32_t lo = 0, hi = 0;
#pragma unroll
    for (int k = 3; k >= 0; --k) {
        const uint64_t x = pair_of(w[k] << 16, w[k] & 0xFFFF0000u);
        const uint64_t n = add_pair(fma_pair(x, p2, snap), whole);
        lo = lo * 16u + static_cast<uint32_t>(n);
        hi = hi * 16u + static_cast<uint32_t>(n >> 32);
    }
    constexpr uint32_t kBits = 0x4B400000u;   // of 1.5 2^23
    return (lo - kBits * 0x1111u) | (hi - kBits * 0x1111u) << 16;
}

// Lanes 0 to 27 have a group each, dims 16 l .., and every lane a pair of the rotated dims.
__global__ void __launch_bounds__(kQ4Warps * 32, 2048 / (kQ4Warps * 32))
    q4_append_kernel(const PagedBatch b, const uint4 *kv, uint8_t *pages, int32_t *status) {
    wait_before();
    const int lane = threadIdx.x & 31;
    const int64_t r = int64_t{blockIdx.x} * kQ4Warps + (threadIdx.x >> 5);
    report_bad(b, status);
    if (r >= b.n_new) return;
    const bool group = lane < kQ4Dims / 16;
    const uint4 *src = kv + r * (kD / 8) + 2 * lane;
    uint4 v0 = {}, v1 = {};
    if (group) {
        v0 = __ldg(src);
        v1 = __ldg(src + 1);
    }
    uint32_t pair =
        __ldg(reinterpret_cast<const uint32_t *>(kv + r * (kD / 8)) + kQ4Dims / 2 + lane);
    int s;
    int32_t p;
    if (!find_row(b, r, lane, s, p)) return;
    uint8_t *row = row_of(b, pages, s, p, lane, status);
    if (!row) return;
    const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
    // the group's largest magnitude (NaN with a NaN among them) as the bits of an fp32: whole
    // numbers in the same order, NaN above all
    uint32_t m2 = w[0];
#pragma unroll
    for (int k = 1; k < 8; ++k)
        asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m2) : "r"(w[k]));
    const uint32_t amax = max((m2 << 16) & 0x7FFF0000u, m2 & 0x7FFF0000u);
    const bool finite = amax < kQ4Limit;
    const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, finite ? amax : 0u);
    const int e = max(static_cast<int>(top >> 23) - 127, kQ4LeastExp);
    const float up = pow2(10 - e);
    // 0 <= amax 2^-E / 7 < 293; the division's rounding never meets a border of e4m3 (amax has
    // eight significant bits, seven times a border as well)
    const uint32_t scale =
        finite ? __nv_cvt_float_to_fp8(__uint_as_float(amax) * up / 7.0f, __NV_SATFINITE,
                                       __NV_E4M3)
               : 0x7Fu;
    const float unit = finite ? e4m3(scale) : 0.0f;
    const float per = unit > 0.0f ? 1.0f / unit : 0.0f;
    // Ordinary rows: the power of two goes into 1 / s, and a normal s (off by 2^-4 at most) leaves
    // no quotient above 7.5.
    const bool plain = __all_sync(0xFFFFFFFFu, finite && (scale >= 8 || scale == 0)) && e > -50 &&
                       e < 70;
    if (group) {
        uint32_t code[2] = {0, 0};
        if (plain) {
            code[0] = eight_plain(w, up * per);
            code[1] = eight_plain(w + 4, up * per);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                code[k / 4] |= whole_plus8(bf16lo(w[k]) * up, per, finite) << (4 * (k % 4));
                code[k / 4] |= whole_plus8(bf16hi(w[k]) * up, per, finite) << (4 * (k % 4) + 16);
            }
        }
        *reinterpret_cast<uint2 *>(row + 32 + 8 * lane) = make_uint2(code[0], code[1]);
    }
    if (b.cos_sin) {
        const float2 a =
            __ldg(reinterpret_cast<const float2 *>(b.cos_sin + int64_t{p} * kRope) + lane);
        pair = turn_pair(pair, a.x, a.y);
    }
    reinterpret_cast<uint32_t *>(row + kQ4Rope)[lane] = pair;
    // the first 32 bytes: chunk lane / 4, half (lane / 2) % 2, group lane % 2 of the half
    const int half = group ? (lane >> 1) & 1 : lane & 1;
    const int at = group ? 2 * (lane >> 2) + (lane & 1) : lane < 30 ? 14 : 15;
    row[16 * half + at] = static_cast<uint8_t>(group ? scale : lane < 30 ? e + 127 : 0);
}

// Lane l has dims 8 l .. and (lanes 0 to 23) 256 + 8 l ..: words l and l + 32 of the codes; and a
// pair of the rotated dims.
__global__ void __launch_bounds__(kQ4Warps * 32)
    q4_read_kernel(const PagedBatch b, uint8_t *pages, uint4 *out, int32_t *status) {
    wait_before();
    const int lane = threadIdx.x & 31;
    const int64_t r = int64_t{blockIdx.x} * kQ4Warps + (threadIdx.x >> 5);
    report_bad(b, status);
    if (r >= b.n_new) return;
    int s;
    int32_t p;
    if (!find_row(b, r, lane, s, p)) return;
    const uint8_t *row = row_of(b, pages, s, p, lane, status);
    if (!row) return;
    const bool more = lane < kQ4Dims / 8 - 32;
    const uint32_t first = __ldg(reinterpret_cast<const uint32_t *>(row + 32) + lane);
    uint32_t second = 0;
    if (more) second = __ldg(reinterpret_cast<const uint32_t *>(row + 32) + 32 + lane);
    uint32_t pair = __ldg(reinterpret_cast<const uint32_t *>(row + kQ4Rope) + lane);
    const uint32_t head = __ldg(row + lane);   // the scales, a byte a lane
    const uint32_t exponent = __shfl_sync(0xFFFFFFFFu, head, 14);
    auto words = [&](uint32_t code, int word) {
        // chunk word / 8, half word / 4 % 2, group word / 2 % 2
        const uint32_t scale = __shfl_sync(0xFFFFFFFFu, head,
                                           (16 * ((word >> 2) & 1) + 2 * (word >> 3) +
                                            ((word >> 1) & 1)) & 31);
        const float u = q4_unit(scale, exponent);
        const __nv_bfloat162 half = __float2bfloat162_rn(0.5f * u);
        const __nv_bfloat162 off = __float2bfloat162_rn(-72.0f * u);
        return make_uint4(q4_pair(code, 0, half, off), q4_pair(code, 1, half, off),
                          q4_pair(code, 2, half, off), q4_pair(code, 3, half, off));
    };
    const uint4 v0 = words(first, lane);
    const uint4 v1 = words(second, lane + 32);
    if (b.cos_sin) {
        const float2 a =
            __ldg(reinterpret_cast<const float2 *>(b.cos_sin + int64_t{p} * kRope) + lane);
        pair = turn_pair(pair, a.x, -a.y);
    }
    uint4 *dst = out + r * (kD / 8);
    dst[lane] = v0;
    if (more) dst[32 + lane] = v1;
    reinterpret_cast<uint32_t *>(dst)[kQ4Dims / 2 + lane] = pair;
}

}  // namespace
}  // namespace dsa

extern "C" int dsa_paged_q4_append(const void *kv, int64_t n_new, const int32_t *new_start,
                                   const int32_t *seq_len, int32_t n_seqs,
                                   const int32_t *page_table, int32_t max_pages, void *pages,
                                   int64_t n_pages, int64_t page_stride, int32_t page_size,
                                   const float *cos_sin, int64_t n_pos, int32_t *dev_status,
                                   void *stream) {
    using namespace dsa;
    if (!kv || !aligned16(kv) || !aligned4(dev_status)) return DSA_ERR_ARG;
    PagedBatch b;
    const int rc = check_paged_batch(n_new, new_start, seq_len, n_seqs, page_table, max_pages,
                                     pages, n_pages, page_stride, page_size, cos_sin, n_pos, &b,
                                     kQ4PageRow);
    if (rc != DSA_OK) return rc;
    if (touches_pages(b, pages, kv, static_cast<uint64_t>(n_new) * kD * 2, kQ4PageRow))
        return DSA_ERR_ARG;
    const unsigned grid = static_cast<unsigned>((n_new + kQ4Warps - 1) / kQ4Warps);
    return launch_overlapped(q4_append_kernel, grid, kQ4Warps * 32, 0,
                             static_cast<cudaStream_t>(stream), b, static_cast<const uint4 *>(kv),
                             static_cast<uint8_t *>(pages), dev_status);
}

extern "C" int dsa_paged_q4_read(const int32_t *new_start, const int32_t *seq_len, int32_t n_seqs,
                                 const int32_t *page_table, int32_t max_pages, const void *pages,
                                 int64_t n_pages, int64_t page_stride, int32_t page_size,
                                 const float *cos_sin, int64_t n_pos, void *out, int64_t n_new,
                                 int32_t *dev_status, void *stream) {
    using namespace dsa;
    if (!out || !aligned16(out) || !aligned4(dev_status)) return DSA_ERR_ARG;
    PagedBatch b;
    const int rc = check_paged_batch(n_new, new_start, seq_len, n_seqs, page_table, max_pages,
                                     pages, n_pages, page_stride, page_size, cos_sin, n_pos, &b,
                                     kQ4PageRow);
    if (rc != DSA_OK) return rc;
    if (touches_pages(b, pages, out, static_cast<uint64_t>(n_new) * kD * 2, kQ4PageRow))
        return DSA_ERR_ARG;
    const unsigned grid = static_cast<unsigned>((n_new + kQ4Warps - 1) / kQ4Warps);
    return launch_overlapped(q4_read_kernel, grid, kQ4Warps * 32, 0,
                             static_cast<cudaStream_t>(stream), b,
                             static_cast<uint8_t *>(const_cast<void *>(pages)),
                             static_cast<uint4 *>(out), dev_status);
}
