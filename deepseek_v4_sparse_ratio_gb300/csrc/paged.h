// The paged KV cache of a ragged batch, as the append and the attention over it see it:
// the arguments both calls share, their checks, and the rule that says which sequences of
// the batch take part.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "common.cuh"

namespace dsa {

constexpr int kRope = DSA_ROPE_DIM;           // rotated elements at the end of a row
constexpr int kRopePairs = DSA_ROPE_DIM / 2;

struct PagedBatch {
    const int32_t *new_start;   // [n_seqs + 1] first row of each sequence's new tokens
    const int32_t *seq_len;     // [n_seqs] tokens of each sequence, the new ones included
    const int32_t *page_table;  // [n_seqs, max_pages]
    const float *cos_sin;       // [n_pos, 32, 2] or null
    int64_t n_new;              // rows of the new tokens' arrays
    int64_t page_stride;        // elements (bytes where a row is in 4 bits)
    int32_t n_seqs, max_pages;
    int32_t n_pages;
    int32_t page_shift;         // log2(rows of a page)
    int32_t len_limit;          // longest sequence the table (and cos_sin) can hold
};

// A row of the pages as their stride counts it: `size` units of `unit` bytes; pages begin on
// multiples of `align` bytes.
struct PageRow {
    int32_t size, unit, align;
};
constexpr PageRow kBf16Row = {kD, 2, 16};
constexpr PageRow kQ4PageRow = {DSA_Q4_ROW_BYTES, 1, 32};  // (read in sectors)

// Checks the arguments that say which rows belong to which sequence at which positions, and fills
// that part of `b` (a sequence may be as long as there are angles, or DSA_MAX_PAGED_TOKENS); DSA_OK
// or a DSA_ERR_* code.
int check_batch(int64_t n_new, const int32_t *new_start, const int32_t *seq_len, int32_t n_seqs,
                const float *cos_sin, int64_t n_pos, PagedBatch *b);

// Checks every argument the paged calls share and fills `b`; DSA_OK or a DSA_ERR_* code.
int check_paged_batch(int64_t n_new, const int32_t *new_start, const int32_t *seq_len,
                      int32_t n_seqs, const int32_t *page_table, int32_t max_pages,
                      const void *pages, int64_t n_pages, int64_t page_stride, int32_t page_size,
                      const float *cos_sin, int64_t n_pos, PagedBatch *b,
                      PageRow row = kBf16Row);

// Whether [p, p + bytes) touches a page (between pages lies what the caller likes).
bool touches_pages(const PagedBatch &b, const void *pages, const void *p, uint64_t bytes,
                   PageRow row = kBf16Row);

inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Whether [a, a + na) and [b, b + nb) share a byte.
inline bool overlaps(const void *a, uint64_t na, const void *b, uint64_t nb) {
    const uint64_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

// The rows of the pages in bf16 elements, boxes of 64 (or 32) of them by the rows of a page (128 at
// most), swizzled over their 128 (64) bytes.
bool make_tmap_pages(CUtensorMap *map, const void *pages, const PagedBatch &b,
                     PageRow row = kBf16Row, uint32_t box_inner = 64);

// One sequence of the batch: rows [row0, row0 + n) are its new tokens, the last n of its len.
struct PagedSeq {
    int32_t row0, n, len;
};

// Sequence s of the batch. A sequence whose numbers contradict each other or the arrays'
// sizes gets n = 0, so nothing of it is read or written; `bad` tells it from an idle one.
__device__ __forceinline__ PagedSeq paged_seq(const PagedBatch &b, int s, bool &bad) {
    const int32_t r0 = __ldg(b.new_start + s), r1 = __ldg(b.new_start + s + 1);
    const int32_t len = __ldg(b.seq_len + s);
    bad = r0 < 0 || r1 < r0 || r1 > b.n_new || len < r1 - r0 || len > b.len_limit;
    return PagedSeq{r0, bad ? 0 : r1 - r0, len};
}

// The sequence that holds row r: the last s with new_start[s] <= r (0 when there is none).
// One round looks at 32 evenly spaced entries, so 1,024 sequences take two rounds.
__device__ __forceinline__ int find_seq(const PagedBatch &b, int64_t r, int lane) {
    int lo = 0, hi = b.n_seqs;  // new_start[lo] <= r (taken for lo = 0), r < new_start[hi]
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) >> 5;
        const int s = lo + lane * step;
        const bool le = s < hi && __ldg(b.new_start + s) <= r;
        const uint32_t m = __ballot_sync(0xFFFFFFFFu, le) | 1u;
        const int k = 31 - __clz(m);
        lo += k * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

__device__ __forceinline__ bool holds(const PagedSeq &q, int64_t r) {
    return r >= q.row0 && r < int64_t{q.row0} + q.n;
}

// The same by looking at every sequence: the last one that holds row r, -1 when none does. For
// rows of padding, and for starts that decrease somewhere, among which find_seq may miss the
// sequence whose numbers are right.
__device__ __forceinline__ int find_seq_any(const PagedBatch &b, int64_t r, int lane) {
    int at = -1;
#pragma unroll 1
    for (int s = lane; s < b.n_seqs; s += 32) {
        bool bad;
        if (holds(paged_seq(b, s, bad), r)) at = s;
    }
    return __reduce_max_sync(0xFFFFFFFFu, at);
}

// A pair (x, y) turned by an angle, in fp32 and rounded to bf16 once.
__device__ __forceinline__ uint32_t turn_pair(uint32_t v, float c, float s) {
    const float x = bf16lo(v), y = bf16hi(v);
    const __nv_bfloat162 r = __floats2bfloat162_rn(x * c - y * s, x * s + y * c);
    return *reinterpret_cast<const uint32_t *>(&r);
}

// What a kernel needs once per device: the raised shared-memory limit, and that it was compiled to
// the registers its warps' split counts on.
template <typename... Args>
int prepare_kernel(void (*kernel)(Args...), int regs, int smem) {
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, kernel) == cudaSuccess && fa.numRegs == regs &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) ==
            cudaSuccess)
        return DSA_OK;
    (void)cudaGetLastError();  // the caller has the code; its own next call is not to find it
    return DSA_ERR_CUDA;
}

// For kernels launched by launch_overlapped: waits until the kernels before this one in the
// stream are done and their writes can be read.
__device__ __forceinline__ void wait_before() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// A launch whose CTAs may be placed as those of the kernel before it in the stream exit (all of
// this library's kernels that it launches begin with wait_before): hides the launch and what a
// kernel sets up before it. (The kernel before could let it be placed earlier still; the join of
// an attention then measured 6 to 12 us later.)
template <typename... Args>
int launch_overlapped(void (*kernel)(Args...), unsigned grid, unsigned threads, size_t smem,
                      cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
        (void)cudaGetLastError();
        return DSA_ERR_CUDA;
    }
    return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace dsa
