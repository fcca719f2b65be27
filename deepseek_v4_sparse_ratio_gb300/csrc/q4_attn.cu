// dsa_paged_q4_attn: attention of a ragged batch's new tokens over their sequences' rows in pages
// of 4-bit rows, all of them or a sliding window and the first few.
//
//   out[r,h] = R(-t) sum_u p_u v_u,   p = softmax_u(scale * (R(t) q[r,h]) . v_u)
//
// The simplest form: a warp per row of q, one key after the other, lane l with dims 16 l ...
#include <math.h>

#include "paged.h"
#include "q4.h"

namespace dsa {

namespace {

struct Q4Args {
    PagedBatch b;
    const uint4 *q;
    const uint8_t *pages;
    uint4 *out;
    int32_t heads, window, sinks, q_turned;
    float c;   // scale log2(e)
    int32_t *status;
};

__device__ __forceinline__ void turn16(float *x, const float *cs, float sign) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float c = __ldg(cs + 2 * k), s = sign * __ldg(cs + 2 * k + 1);
        const float a = x[2 * k] * c - x[2 * k + 1] * s;
        x[2 * k + 1] = x[2 * k] * s + x[2 * k + 1] * c;
        x[2 * k] = a;
    }
}

__device__ __forceinline__ void floats16(const uint4 &a, const uint4 &b, float *x) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        x[2 * k] = bf16lo(w[k]);
        x[2 * k + 1] = bf16hi(w[k]);
    }
}

__global__ void __launch_bounds__(256) q4_attn_kernel(const __grid_constant__ Q4Args p) {
    wait_before();
    const int lane = threadIdx.x & 31;
    const int64_t item = int64_t{blockIdx.x} * 8 + (threadIdx.x >> 5);
    if (blockIdx.x == 0) {
        for (int s = threadIdx.x; s < p.b.n_seqs; s += blockDim.x) {
            bool bad;
            paged_seq(p.b, s, bad);
            if (bad) report(p.status, DSA_ERR_BOUNDS);
        }
    }
    const int64_t r = item / p.heads;
    if (r >= p.b.n_new) return;
    const int s = find_seq_any(p.b, r, lane);
    if (s < 0) return;
    bool bad;
    const PagedSeq sq = paged_seq(p.b, s, bad);
    const int t = sq.len - sq.n + static_cast<int>(r - sq.row0);
    const float *cs = p.b.cos_sin && lane >= 28
                          ? p.b.cos_sin + int64_t{t} * kRope + 16 * (lane - 28)
                          : nullptr;
    float q[16], o[16];
    floats16(p.q[item * 64 + 2 * lane], p.q[item * 64 + 2 * lane + 1], q);
    if (cs && !p.q_turned) turn16(q, cs, 1.0f);
#pragma unroll
    for (int k = 0; k < 16; ++k) o[k] = 0.0f;
    float m = -INFINITY, sum = 0.0f;
    const int low = p.window > 0 ? max(0, t - p.window + 1) : 0;
    const int sinks = min(p.sinks, low);
    for (int j = 0; j < sinks + t + 1 - low; ++j) {
        const int u = j < sinks ? j : low + j - sinks;
        const int32_t page = __ldg(p.b.page_table + int64_t{s} * p.b.max_pages +
                                   (u >> p.b.page_shift));
        if (page < 0 || page >= p.b.n_pages) {
            if (lane == 0) report(p.status, DSA_ERR_BOUNDS);
            continue;
        }
        const uint8_t *row = p.pages + page * p.b.page_stride +
                             int64_t{u & ((1 << p.b.page_shift) - 1)} * kQ4Row;
        float x[16];
        if (lane >= 28) {
            const uint4 *at = reinterpret_cast<const uint4 *>(row + kQ4Rope) + 2 * (lane - 28);
            floats16(__ldg(at), __ldg(at + 1), x);
        } else {
            const uint2 w = __ldg(reinterpret_cast<const uint2 *>(row + 32) + lane);
            const float unit = q4_unit(
                __ldg(row + 16 * ((lane >> 1) & 1) + 2 * (lane >> 2) + (lane & 1)),
                __ldg(row + 14));
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const uint32_t word = k < 8 ? w.x : w.y;
                const int at = 4 * (k % 8 / 2) + 16 * (k & 1);
                x[k] = (static_cast<int>((word >> at) & 15u) - 8) * unit;
            }
        }
        float dot = 0.0f;
#pragma unroll
        for (int k = 0; k < 16; ++k) dot = fmaf(q[k], x[k], dot);
#pragma unroll
        for (int k = 16; k >= 1; k >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, k);
        const float m_new = fmaxf(m, dot);
        const float alpha = m == m_new ? 1.0f : exp2f((m - m_new) * p.c);
        const float w = dot == -INFINITY ? 0.0f : exp2f((dot - m_new) * p.c);
        m = m_new;
        sum = sum * alpha + w;
#pragma unroll
        for (int k = 0; k < 16; ++k) o[k] = o[k] * alpha + w * x[k];
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int k = 0; k < 16; ++k) o[k] *= inv;
    if (cs) turn16(o, cs, -1.0f);
    uint32_t w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(o[2 * k], o[2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t *>(&v);
    }
    p.out[item * 64 + 2 * lane] = make_uint4(w[0], w[1], w[2], w[3]);
    p.out[item * 64 + 2 * lane + 1] = make_uint4(w[4], w[5], w[6], w[7]);
}

}  // namespace
}  // namespace dsa

extern "C" int dsa_paged_q4_attn(const void *q, int32_t heads, int64_t n_new,
                                 const int32_t *new_start, const int32_t *seq_len, int32_t n_seqs,
                                 const int32_t *page_table, int32_t max_pages, const void *pages,
                                 int64_t n_pages, int64_t page_stride, int32_t page_size,
                                 const float *cos_sin, int64_t n_pos, int32_t window,
                                 int32_t sinks, int32_t q_turned, float scale, void *workspace,
                                 size_t workspace_bytes, void *out, int32_t *dev_status,
                                 void *stream) {
    using namespace dsa;
    if (!q || !out || !aligned16(q) || !aligned16(out) || !aligned4(dev_status))
        return DSA_ERR_ARG;
    Q4Args p;
    const int rc = check_paged_batch(n_new, new_start, seq_len, n_seqs, page_table, max_pages,
                                     pages, n_pages, page_stride, page_size, cos_sin, n_pos, &p.b,
                                     kQ4PageRow);
    if (rc != DSA_OK) return rc;
    const float c = scale * 1.4426950408889634f;
    if (heads < 1 || heads > DSA_MAX_PAGED_HEADS || window < 0 || sinks < 0 ||
        sinks > DSA_MAX_SINKS || q_turned < 0 || q_turned > 1 || !(scale > 0.0f) || isinf(c) ||
        n_new * heads > (int64_t{1} << 31) - 1)
        return DSA_ERR_SHAPE;
    const uint64_t bytes = static_cast<uint64_t>(n_new) * heads * kD * 2;
    const uint64_t used = DSA_PAGED_WORKSPACE_BYTES;
    if (overlaps(q, bytes, out, bytes) || touches_pages(p.b, pages, out, bytes, kQ4PageRow))
        return DSA_ERR_ARG;
    if (!workspace || !aligned16(workspace) || workspace_bytes < used) return DSA_ERR_SCRATCH;
    if (overlaps(workspace, used, q, bytes) || overlaps(workspace, used, out, bytes) ||
        touches_pages(p.b, pages, workspace, used, kQ4PageRow))
        return DSA_ERR_ARG;
    p.q = static_cast<const uint4 *>(q);
    p.pages = static_cast<const uint8_t *>(pages);
    p.out = static_cast<uint4 *>(out);
    p.heads = heads;
    p.window = window;
    p.sinks = window > 0 ? sinks : 0;
    p.q_turned = q_turned;
    p.c = c;
    p.status = dev_status;
    return launch_overlapped(q4_attn_kernel, static_cast<unsigned>((n_new * heads + 7) / 8), 256, 0,
                             static_cast<cudaStream_t>(stream), p);
}
