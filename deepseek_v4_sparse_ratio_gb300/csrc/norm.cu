// dsa_qk_norm_rope: the new tokens' query heads and KV rows, normalised and rotated in one pass.
//
//   y = R(p) (x rsqrt(mean x^2 + eps) w)
//
// A row (a head of q, or a KV row) is 512 elements, 16 of a lane: pieces l and l + 32 of 16 bytes,
// so that the rotated dims are the second pieces of lanes 24..31. A warp takes up to four heads of
// a token, whose place and angles it looks up once; a token's KV row is a warp's own.
// Bound by HBM: 4,096 tokens of 64 heads (545 MB) take 78.6 us, 1.04 of the copy rate (the last
// 50 MB of the output are still in L2 then); one token takes 8 us, the launch's.
#include <math.h>

#include "common.cuh"
#include "paged.h"

namespace dsa {

namespace {

constexpr int kNormWarps = 8;
constexpr int kNormRows = 4;  // heads of a token that a warp takes, all their loads in flight

struct NormArgs {
    PagedBatch b;             // (no pages)
    const uint4 *q, *kv;
    uint4 *q_out, *kv_out;
    const float *q_weight, *kv_weight;
    float eps;
    int32_t heads;
    int32_t groups;           // of heads, and one for the KV row
    int32_t *status;
};

__device__ __forceinline__ float square_sum(uint4 v, float s) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        s = fmaf(bf16lo(w[k]), bf16lo(w[k]), s);
        s = fmaf(bf16hi(w[k]), bf16hi(w[k]), s);
    }
    return s;
}

// Eight elements times r and their weights, four pairs turned by cs (or not), rounded once.
__device__ __forceinline__ uint4 scaled8(uint4 v, float r, const float *w, bool weights,
                                         const float4 *cs) {
    uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float a = bf16lo(x[k]) * r, b = bf16hi(x[k]) * r;
        if (weights) {
            a *= w[2 * k];
            b *= w[2 * k + 1];
        }
        if (cs) {
            const float c = k & 1 ? cs[k / 2].z : cs[k / 2].x;
            const float s = k & 1 ? cs[k / 2].w : cs[k / 2].y;
            const float t = a * c - b * s;
            b = a * s + b * c;
            a = t;
        }
        const __nv_bfloat162 y = __floats2bfloat162_rn(a, b);
        x[k] = *reinterpret_cast<const uint32_t *>(&y);
    }
    return make_uint4(x[0], x[1], x[2], x[3]);
}

__global__ void __launch_bounds__(kNormWarps * 32)
    qk_norm_rope_kernel(const __grid_constant__ NormArgs p) {
    wait_before();
    const int lane = threadIdx.x & 31;
    const int64_t item = int64_t{blockIdx.x} * kNormWarps + (threadIdx.x >> 5);
    if (blockIdx.x == 0) {
        for (int s = threadIdx.x; s < p.b.n_seqs; s += blockDim.x) {
            bool bad;
            paged_seq(p.b, s, bad);
            if (bad) report(p.status, DSA_ERR_BOUNDS);
        }
    }
    const int64_t r = item / p.groups;
    if (r >= p.b.n_new) return;
    const int g = static_cast<int>(item - r * p.groups);
    const bool of_kv = g == p.groups - 1;
    const int n = of_kv ? 1 : min(kNormRows, p.heads - g * kNormRows);
    const int64_t at = (of_kv ? r : r * p.heads + g * kNormRows) * (kD / 8) + lane;
    // (in place: a row is read and written by one warp alone)
    const uint4 *src = (of_kv ? p.kv : p.q) + at;
    uint4 *dst = (of_kv ? p.kv_out : p.q_out) + at;
    uint4 v[kNormRows][2];
#pragma unroll
    for (int i = 0; i < kNormRows; ++i)
        if (i < n) {
            v[i][0] = src[i * (kD / 8)];
            v[i][1] = src[i * (kD / 8) + 32];
        }
    int s = find_seq(p.b, r, lane);
    bool bad;
    PagedSeq q = paged_seq(p.b, s, bad);
    if (!holds(q, r)) {
        s = find_seq_any(p.b, r, lane);
        if (s < 0) return;
        q = paged_seq(p.b, s, bad);
    }
    const int32_t pos = q.len - q.n + static_cast<int32_t>(r - q.row0);
    float4 cs[2];
    const bool turn = p.b.cos_sin && lane >= 24;
    if (turn) {
        const float4 *from =
            reinterpret_cast<const float4 *>(p.b.cos_sin + int64_t{pos} * kRope) + (lane - 24) * 2;
        cs[0] = __ldg(from);
        cs[1] = __ldg(from + 1);
    }
    const float *weight = of_kv ? p.kv_weight : p.q_weight;
    float w[16];
    if (weight) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float4 x = __ldg(reinterpret_cast<const float4 *>(weight) + (k / 2) * 64 +
                                   2 * lane + (k & 1));
            w[4 * k] = x.x;
            w[4 * k + 1] = x.y;
            w[4 * k + 2] = x.z;
            w[4 * k + 3] = x.w;
        }
    }
#pragma unroll
    for (int i = 0; i < kNormRows; ++i) {
        if (i >= n) break;
        float sum = square_sum(v[i][1], square_sum(v[i][0], 0.0f));
#pragma unroll
        for (int k = 16; k >= 1; k >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, k);
        const float f = 1.0f / sqrtf(sum * (1.0f / kD) + p.eps);
        dst[i * (kD / 8)] = scaled8(v[i][0], f, w, weight != nullptr, nullptr);
        dst[i * (kD / 8) + 32] =
            scaled8(v[i][1], f, w + 8, weight != nullptr, turn ? cs : nullptr);
    }
}

}  // namespace
}  // namespace dsa

extern "C" int dsa_qk_norm_rope(const void *q, int32_t heads, const void *kv, int64_t n_new,
                                const int32_t *new_start, const int32_t *seq_len, int32_t n_seqs,
                                const float *q_weight, const float *kv_weight, float eps,
                                const float *cos_sin, int64_t n_pos, void *q_out, void *kv_out,
                                int32_t *dev_status, void *stream) {
    using namespace dsa;
    if (!q || !kv || !q_out || !kv_out || !aligned16(q) || !aligned16(kv) || !aligned16(q_out) ||
        !aligned16(kv_out) || !aligned16(q_weight) || !aligned16(kv_weight) ||
        !aligned4(dev_status))
        return DSA_ERR_ARG;
    NormArgs p = {};
    int rc = check_batch(n_new, new_start, seq_len, n_seqs, cos_sin, n_pos, &p.b);
    if (rc != DSA_OK) return rc;
    if (heads < 1 || heads > DSA_MAX_PAGED_HEADS || !(eps > 0.0f) || isinf(eps) ||
        n_new * heads > (int64_t{1} << 31) - 1)
        return DSA_ERR_SHAPE;
    const uint64_t kv_bytes = static_cast<uint64_t>(n_new) * kD * 2, q_bytes = kv_bytes * heads;
    if ((q_out != q && overlaps(q_out, q_bytes, q, q_bytes)) ||
        (kv_out != kv && overlaps(kv_out, kv_bytes, kv, kv_bytes)) ||
        overlaps(q_out, q_bytes, kv, kv_bytes) || overlaps(kv_out, kv_bytes, q, q_bytes) ||
        overlaps(q_out, q_bytes, kv_out, kv_bytes))
        return DSA_ERR_ARG;
    p.q = static_cast<const uint4 *>(q);
    p.kv = static_cast<const uint4 *>(kv);
    p.q_out = static_cast<uint4 *>(q_out);
    p.kv_out = static_cast<uint4 *>(kv_out);
    p.q_weight = q_weight;
    p.kv_weight = kv_weight;
    p.eps = eps;
    p.heads = heads;
    p.groups = (heads + kNormRows - 1) / kNormRows + 1;
    p.status = dev_status;
    const int64_t grid = (n_new * p.groups + kNormWarps - 1) / kNormWarps;
    return launch_overlapped(qk_norm_rope_kernel, static_cast<unsigned>(grid), kNormWarps * 32, 0,
                             static_cast<cudaStream_t>(stream), p);
}
