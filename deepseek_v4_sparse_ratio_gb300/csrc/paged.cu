// dsa_paged_append: new KV rows of a ragged batch into a paged cache, their position
// rotation applied on the way; and the argument checks it shares with dsa_paged_attn.
//
// Row r of sequence s (the one with new_start[s] <= r < new_start[s+1]) has position
// p = seq_len[s] - n_s + (r - new_start[s]) and goes to row p mod page_size of page
// page_table[s][p / page_size]. Pairs (x, y) = elements (448 + 2i, 449 + 2i) become
// (x c - y s, x s + y c) with (c, s) = cos_sin[p][i], in fp32 and rounded to bf16 once; the
// other 448 elements are copied. Bound by HBM (a row in, a row out, 256 bytes of angles): 56,436
// rows of 16 sequences in 20.1 us, 0.95 of the measured copy rate; up to a few thousand rows
// by the launch (4 us). One warp per row: the row's loads are in flight while its sequence is
// looked up.
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "paged.h"

namespace dsa {

namespace {

constexpr int kAppendWarps = 8;

// One warp per row; lane l moves 16-byte pieces l and l + 32, and the last eight pieces
// hold the rotated pairs. The bound keeps it at 32 registers, eight CTAs an SM (with 38, six
// CTAs: 25.6 instead of 23.6 us for 56,436 rows from a cold L2).
__global__ void __launch_bounds__(kAppendWarps * 32, 2048 / (kAppendWarps * 32))
    paged_append_kernel(const PagedBatch b, const uint4 *kv, __nv_bfloat16 *pages,
                        int32_t *status) {
    wait_before();
    const int lane = threadIdx.x & 31;
    const int64_t r = int64_t{blockIdx.x} * kAppendWarps + (threadIdx.x >> 5);
    if (blockIdx.x == 0) {
        for (int s = threadIdx.x; s < b.n_seqs; s += blockDim.x) {
            bool bad;
            paged_seq(b, s, bad);
            if (bad) report(status, DSA_ERR_BOUNDS);
        }
    }
    if (r >= b.n_new) return;
    const uint4 *src = kv + r * (kD / 8) + lane;
    uint4 v0 = __ldg(src), v1 = __ldg(src + 32);
    int s = find_seq(b, r, lane);
    bool bad;
    PagedSeq q = paged_seq(b, s, bad);
    if (!holds(q, r)) {
        s = find_seq_any(b, r, lane);
        if (s < 0) return;
        q = paged_seq(b, s, bad);
    }
    const int32_t p = q.len - q.n + static_cast<int32_t>(r - q.row0);
    const int32_t page = __ldg(b.page_table + int64_t{s} * b.max_pages + (p >> b.page_shift));
    if (page < 0 || page >= b.n_pages) {
        if (lane == 0) report(status, DSA_ERR_BOUNDS);
        return;
    }
    if (b.cos_sin && lane >= 24) {
        const float4 *cs =
            reinterpret_cast<const float4 *>(b.cos_sin + int64_t{p} * kRope) + (lane - 24) * 2;
        const float4 a = __ldg(cs), c = __ldg(cs + 1);
        v1.x = turn_pair(v1.x, a.x, a.y);
        v1.y = turn_pair(v1.y, a.z, a.w);
        v1.z = turn_pair(v1.z, c.x, c.y);
        v1.w = turn_pair(v1.w, c.z, c.w);
    }
    uint4 *dst = reinterpret_cast<uint4 *>(pages + page * b.page_stride +
                                           int64_t{p & ((1 << b.page_shift) - 1)} * kD) +
                 lane;
    dst[0] = v0;
    dst[32] = v1;
}

}  // namespace

int check_batch(int64_t n_new, const int32_t *new_start, const int32_t *seq_len, int32_t n_seqs,
                const float *cos_sin, int64_t n_pos, PagedBatch *b) {
    if (!new_start || !seq_len || n_new <= 0 || n_seqs <= 0) return DSA_ERR_ARG;
    if (!aligned4(new_start) || !aligned4(seq_len) || !aligned16(cos_sin)) return DSA_ERR_ARG;
    if (cos_sin && n_pos <= 0) return DSA_ERR_ARG;
    // the kernels' walks over the sequences step past the last one, in 32 bits
    if (n_new > (int64_t{1} << 31) - 1 || n_seqs > DSA_MAX_PAGED_SEQS) return DSA_ERR_SHAPE;
    b->new_start = new_start;
    b->seq_len = seq_len;
    b->cos_sin = cos_sin;
    b->n_new = n_new;
    b->n_seqs = n_seqs;
    int64_t len = DSA_MAX_PAGED_TOKENS;
    if (cos_sin) len = std::min(len, n_pos);
    b->len_limit = static_cast<int32_t>(len);
    return DSA_OK;
}

int check_paged_batch(int64_t n_new, const int32_t *new_start, const int32_t *seq_len,
                      int32_t n_seqs, const int32_t *page_table, int32_t max_pages,
                      const void *pages, int64_t n_pages, int64_t page_stride, int32_t page_size,
                      const float *cos_sin, int64_t n_pos, PagedBatch *b, PageRow row) {
    // (null pointers, counts and alignments of all arguments before any limit)
    if (!page_table || !pages || max_pages <= 0 || n_pages <= 0) return DSA_ERR_ARG;
    if (!aligned4(page_table) || reinterpret_cast<uintptr_t>(pages) % row.align != 0)
        return DSA_ERR_ARG;
    const int rc = check_batch(n_new, new_start, seq_len, n_seqs, cos_sin, n_pos, b);
    if (rc != DSA_OK) return rc;
    if (page_size < 16 || page_size > DSA_MAX_PAGE_SIZE || (page_size & (page_size - 1)) != 0)
        return DSA_ERR_SHAPE;
    // a page stride is a byte stride of the tensor map: a multiple of 16 (32) below 2^40
    if (page_stride < int64_t{page_size} * row.size || page_stride % (row.align / row.unit) != 0 ||
        page_stride >= (int64_t{1} << 39))
        return DSA_ERR_SHAPE;
    const int64_t limit = (int64_t{1} << 31) - 1;
    if (n_pages > limit || int64_t{max_pages} * page_size > limit) return DSA_ERR_SHAPE;
    b->page_table = page_table;
    b->page_stride = page_stride;
    b->max_pages = max_pages;
    b->n_pages = static_cast<int32_t>(n_pages);
    b->page_shift = 0;
    while ((1 << b->page_shift) < page_size) ++b->page_shift;
    b->len_limit = static_cast<int32_t>(
        std::min(int64_t{max_pages} * page_size, int64_t{b->len_limit}));
    return DSA_OK;
}

bool touches_pages(const PagedBatch &b, const void *pages, const void *p, uint64_t bytes,
                   PageRow row) {
    const uint64_t base = reinterpret_cast<uintptr_t>(pages), at = reinterpret_cast<uintptr_t>(p);
    const uint64_t stride = static_cast<uint64_t>(b.page_stride) * row.unit;
    const uint64_t page = static_cast<uint64_t>(row.size) * row.unit << b.page_shift;
    // the first page that ends behind `at`: does it begin before the end?
    const uint64_t k = at < base + page ? 0 : (at - base - page) / stride + 1;
    return k < static_cast<uint64_t>(b.n_pages) && base + k * stride < at + bytes;
}

}  // namespace dsa

extern "C" int dsa_paged_append(const void *kv, int64_t n_new, const int32_t *new_start,
                                const int32_t *seq_len, int32_t n_seqs, const int32_t *page_table,
                                int32_t max_pages, void *pages, int64_t n_pages,
                                int64_t page_stride, int32_t page_size, const float *cos_sin,
                                int64_t n_pos, int32_t *dev_status, void *stream) {
    using namespace dsa;
    if (!kv || !aligned16(kv) || !aligned4(dev_status)) return DSA_ERR_ARG;
    PagedBatch b;
    int rc = check_paged_batch(n_new, new_start, seq_len, n_seqs, page_table, max_pages, pages,
                               n_pages, page_stride, page_size, cos_sin, n_pos, &b);
    if (rc != DSA_OK) return rc;
    if (touches_pages(b, pages, kv, static_cast<uint64_t>(n_new) * kD * 2)) return DSA_ERR_ARG;
    const unsigned grid = static_cast<unsigned>((n_new + kAppendWarps - 1) / kAppendWarps);
    return launch_overlapped(paged_append_kernel, grid, kAppendWarps * 32, 0,
                             static_cast<cudaStream_t>(stream), b, static_cast<const uint4 *>(kv),
                             static_cast<__nv_bfloat16 *>(pages), dev_status);
}
