// dsa_paged_attn: attention of a ragged batch's new tokens over their sequences' rows in a
// paged cache.
//
// Simplest form: one warp per (token, head) walks the token's keys in order with an online
// softmax in fp32; lane l holds elements 16 l .. 16 l + 15 of the query, the row and the sum.
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "paged.h"

namespace dsa {

namespace {

__device__ __forceinline__ void unpack16(const uint4 a, const uint4 b, float (&x)[16]) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[2 * i] = bf16lo(w[i]);
        x[2 * i + 1] = bf16hi(w[i]);
    }
}

// grid.x: sequences, grid.y: token stride; the warps of a block share a token's heads.
__global__ void __launch_bounds__(256)
    paged_attn_kernel(const PagedBatch b, const uint4 *__restrict__ q, const uint4 *pages,
                      int heads, int window, float c, uint4 *out, int32_t *status) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int s = blockIdx.x;
    bool bad;
    const PagedSeq sq = paged_seq(b, s, bad);
    if (bad && blockIdx.y == 0 && threadIdx.x == 0) report(status, DSA_ERR_BOUNDS);
    const int32_t *table = b.page_table + int64_t{s} * b.max_pages;
    const int64_t units = int64_t{sq.n} * heads;
    for (int64_t u = int64_t{blockIdx.y} * 8 + warp; u < units; u += int64_t{gridDim.y} * 8) {
        const int i = static_cast<int>(u / heads);
        const int32_t t = sq.len - sq.n + i;
        const int64_t row = int64_t{sq.row0} * heads + u;
        float x[16], o[16];
        unpack16(q[row * 64 + 2 * lane], q[row * 64 + 2 * lane + 1], x);
        const float *cs = b.cos_sin ? b.cos_sin + int64_t{t} * kRope + (lane - 28) * 16 : nullptr;
        const bool turn = cs && lane >= 28;
        if (turn) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float a = x[2 * e], d = x[2 * e + 1];
                x[2 * e] = a * cs[2 * e] - d * cs[2 * e + 1];
                x[2 * e + 1] = a * cs[2 * e + 1] + d * cs[2 * e];
            }
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = 0.0f;
        float m = -INFINITY, l = 0.0f;
        for (int32_t k = window > 0 ? max(0, t - window + 1) : 0; k <= t; ++k) {
            const int32_t page = __ldg(table + (k >> b.page_shift));
            if (page < 0 || page >= b.n_pages) {
                if (lane == 0) report(status, DSA_ERR_BOUNDS);
                continue;
            }
            const uint4 *src = pages + page * (b.page_stride / 8) +
                               int64_t{k & ((1 << b.page_shift) - 1)} * 64 + 2 * lane;
            float v[16];
            unpack16(src[0], src[1], v);
            float dot = 0.0f;
#pragma unroll
            for (int e = 0; e < 16; ++e) dot = fmaf(x[e], v[e], dot);
#pragma unroll
            for (int w = 16; w >= 1; w >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, w);
            dot *= c;
            const float mn = fmaxf(m, dot);
            const float a = m == mn ? 1.0f : exp2f(m - mn), p = exp2f(dot - mn);
            m = mn;
            l = l * a + p;
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = fmaf(p, v[e], o[e] * a);
        }
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] *= inv;
        if (turn) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float a = o[2 * e], d = o[2 * e + 1];
                o[2 * e] = a * cs[2 * e] + d * cs[2 * e + 1];
                o[2 * e + 1] = d * cs[2 * e] - a * cs[2 * e + 1];
            }
        }
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const __nv_bfloat162 r = __floats2bfloat162_rn(o[2 * e], o[2 * e + 1]);
            w[e] = *reinterpret_cast<const uint32_t *>(&r);
        }
        out[row * 64 + 2 * lane] = make_uint4(w[0], w[1], w[2], w[3]);
        out[row * 64 + 2 * lane + 1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

}  // namespace
}  // namespace dsa

extern "C" int dsa_paged_attn(const void *q, int32_t heads, int64_t n_new,
                              const int32_t *new_start, const int32_t *seq_len, int32_t n_seqs,
                              const int32_t *page_table, int32_t max_pages, const void *pages,
                              int64_t n_pages, int64_t page_stride, int32_t page_size,
                              const float *cos_sin, int64_t n_pos, int32_t window, float scale,
                              void *workspace, size_t workspace_bytes, void *out,
                              int32_t *dev_status, void *stream) {
    using namespace dsa;
    if (!q || !out || !aligned16(q) || !aligned16(out) ||
        (reinterpret_cast<uintptr_t>(dev_status) & 3u) != 0)
        return DSA_ERR_ARG;
    PagedBatch b;
    int rc = check_paged_batch(n_new, new_start, seq_len, n_seqs, page_table, max_pages, pages,
                               n_pages, page_stride, page_size, cos_sin, n_pos, &b);
    if (rc != DSA_OK) return rc;
    if (heads < 1 || heads > DSA_MAX_PAGED_HEADS || window < 0 || !(scale > 0.0f) ||
        isinf(scale) || n_new * heads > (int64_t{1} << 31) - 1)
        return DSA_ERR_SHAPE;
    const uintptr_t qa = reinterpret_cast<uintptr_t>(q), oa = reinterpret_cast<uintptr_t>(out);
    const uintptr_t bytes = static_cast<uintptr_t>(n_new) * heads * kD * 2;
    if (qa < oa + bytes && oa < qa + bytes) return DSA_ERR_ARG;
    if (!workspace || !aligned16(workspace) || workspace_bytes < DSA_PAGED_WORKSPACE_BYTES)
        return DSA_ERR_SCRATCH;
    const unsigned gy = static_cast<unsigned>(
        std::min<int64_t>((n_new * heads + 7) / 8, std::max(1, 4864 / n_seqs)));
    paged_attn_kernel<<<dim3(n_seqs, gy), 256, 0, static_cast<cudaStream_t>(stream)>>>(
        b, static_cast<const uint4 *>(q), static_cast<const uint4 *>(pages), heads, window,
        scale * 1.4426950408889634f, static_cast<uint4 *>(out), dev_status);
    return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}
