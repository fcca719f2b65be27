// dsa_paged_q4_attn: attention of a ragged batch's new tokens over their sequences' rows in pages
// of 4-bit rows, all of them or a sliding window and the first few.
//
//   out[r,h] = R(-t) sum_u p_u v_u,   p = softmax_u(scale * (R(t) q[r,h]) . v_u)
//
// Units of up to 64 rows of q and blocks of 128 keys, one list of both cut evenly over the SMs and
// joined, as for single tokens over bf16 pages (paged_walk.cuh, paged_attn.cu). A block, keys on
// the MMA's M:
//   S^T[key, row]  = K_blk[128 x 512] . Q^T        (M=128, N=64, K=512)
//   O^T[d, row]   += V_blk^T[512 x 128] . P^T       (4 x (M=128, N=64, K=128))
// in bf16, which holds what a 4-bit element stands for exactly. What binds first is shared memory:
// with both operands there a product of N=64 takes 48 cycles for 32 of the tensor pipe, and the
// unpacked rows are written on top. So six of the eight 64-dim chunks of K are unpacked into TMEM,
// where the first product takes them from (32 cycles), and from there into shared memory when the
// block before has left it; the second product needs them there, transposed. That also takes the
// unpacking and the first product of a block out of the chain: they run beside the softmax and the
// second product of the block before.
//   chunks 0-5: TMEM for QK, shared memory for PV;  chunk 6: shared memory for both, unpacked when
//   PV of the block before has used it (the first tile of PV);  chunk 7, the rotated dims (bf16 in
//   the pages): TMA into their place as soon as the same tile has left it.
// The 4-bit bytes come by TMA too, 64 of a row's first 256 at a time (the scales and chunk 0,
// chunks 1-2, 3-4, 5-6), into two slots in turn. (Loaded by the unpacking threads themselves, a
// key's bytes each, a sector and a line for every lane of a load keep the load unit busy for longer
// than the products take.)
// Measured: 2,048 tokens of 64 heads at 16,384 in 4.63 ms (892 TFLOP/s, 0.45 of the peak); a block
// takes 5,600 cycles there, and the eight unpacking warps are busy through it: that chain is what
// bounds it now, before shared memory and the tensor pipe (2,048 cycles). Shared memory's part by
// bytes, at 128 a cycle: operands of QK 64 + 32 KB and of PV 192 KB, 4-bit bytes in and out 64 KB,
// unpacked rows in 112 KB, chunk 7 and P 16 KB each, 496 KB or 3,970 cycles. (The 128 rows of the
// bf16 chunk kernel share a block's loads among twice the rows: 3.71 ms, and 3.65 ms with the
// context's rows read back first.) One token at 131,072: 41.1 us among other calls, its 50 MB of
// pages in L2 by then; from a cold L2 6 us more. 6,700 cycles a block.
// Between units lie 18,000 cycles (results out, first block's softmax): 285 us for 7 prompts of up
// to 1,701 tokens of 16 heads with a window of 512. The code that is run there is kept in short
// loops: fetching it is most of its time.
//
// Roles (640 threads): warp 0 loads the 4-bit bytes; warp 1 issues QK, warp 3 PV; warp 2 loads q,
// turns it, and loads chunk 7; warps 4-11 unpack: thread = key, each half of the warps every other
// chunk; warps 12-19 softmax and results, 32 rows of 32 keys a warp.
#include <cudaTypedefs.h>
#include <math.h>

#include <algorithm>
#include <mutex>

#include "paged_walk.cuh"
#include "q4.h"

namespace dsa {

namespace {

using namespace paged;

constexpr int kT = 640;
constexpr int kQkWarp = 1;
constexpr int kQWarp = 2;
constexpr int kPvWarp = 3;
constexpr int kUnpackWarp0 = 4;
constexpr int kSoftWarp0 = 12;
constexpr int kRegsLaunch = 96;
constexpr int kRegsLow = 80;
constexpr int kRegsSoft = 120;     // 384*80 + 256*120 = 640*96, the launch allocation

constexpr int kRows = 64;          // rows of q in a unit (MMA N)
constexpr int kRing = 4;           // blocks whose valid keys are kept

// shared memory
constexpr uint32_t kChunk = 16384;                // [128 keys x 64 dims]
constexpr uint32_t kOffQ = 0;                     // 8 chunks x [64 rows x 128 B]
constexpr uint32_t kOffV = 65536;                 // chunks 0-5, for PV
constexpr uint32_t kOff6 = kOffV + 6 * kChunk;    // chunk 6
constexpr uint32_t kOff7 = kOff6 + kChunk;        // chunk 7
constexpr uint32_t kOffRaw = kOff7 + kChunk;      // [2][128 keys x 64 B] of the pages
constexpr uint32_t kOffP = kOffRaw + 16384;       // P^T [128 keys x 64 rows] bf16
constexpr uint32_t kOffRed = kOffP + 16384;       // [4][64] block maxima | partial sums
constexpr uint32_t kOffLinv = kOffRed + 1024;     // [64] rescale factors | 1/sum
constexpr uint32_t kOffM = kOffLinv + 256;        // [2][64] running maxima, negated, in turn
constexpr uint32_t kOffWalk = kOffM + 512;        // [2] where the softmax is, by half
constexpr uint32_t kOffBar = kOffWalk + 2 * 192;
constexpr uint32_t kSmem = kOffBar + 384;
static_assert(kSmem <= 232448, "over the shared memory of one CTA");

// TMEM columns
constexpr uint32_t kOCol = 0;      // O^T: 4 d-tiles x 64
constexpr uint32_t kSCol = 256;    // S^T
constexpr uint32_t kKCol = 320;    // chunks 0-5 of K, 32 columns each

// Where a half of the softmax warps is: its segment and, in turn with it, the next one.
struct SoftWalk {
    Walk walk;
    Segment x[2];
    int more[2];
};
static_assert(sizeof(SoftWalk) <= 192, "walks");

// D[tmem] (+)= A[tmem] * B[smem]^T; A: lane = row, a column holds two bf16 along K.
__device__ __forceinline__ void mma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
        : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
        "%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15])
        : "memory");
}

// Bytes brought to L2.
__device__ __forceinline__ void prefetch_rows(const uint8_t *at, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(at), "r"(bytes) : "memory");
}

// Four words (32 dims) as 16 pairs of bf16. `two`: the scales of their two groups (e4m3, the lower
// 16 bits); half_pow: half of the row's power of two.
__device__ __forceinline__ void unpack32(const uint32_t *w, uint32_t two, float half_pow,
                                         uint32_t *out) {
    const __half2_raw h =
        __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
    const float2 s = __half22float2(__half2(h));
    const __nv_bfloat162 half[2] = {__float2bfloat162_rn(s.x * half_pow),
                                    __float2bfloat162_rn(s.y * half_pow)};
    const __nv_bfloat162 k144 = __float2bfloat162_rn(-144.0f);   // (144 u / 2: eight bits, exact)
    const __nv_bfloat162 off[2] = {__hmul2(half[0], k144), __hmul2(half[1], k144)};
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) out[4 * j + k] = q4_pair(w[j], k, half[j / 2], off[j / 2]);
}

// Whether a byte of a word is an e4m3 NaN (0x7F or 0xFF).
__device__ __forceinline__ bool has_nan(uint32_t w) {
    const uint32_t x = ~w & 0x7F7F7F7Fu;   // a byte 0 where all seven bits are set
    return ((x - 0x01010101u) & ~x & 0x80808080u) != 0;
}

// 16 bytes to shared memory.
__device__ __forceinline__ void store_piece(uint32_t at, const uint32_t *v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3])
                 : "memory");
}

// 16 bytes from shared memory.
__device__ __forceinline__ void load_piece(uint32_t *v, uint32_t at) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(at)
                 : "memory");
}

// Hands bytes of shared memory that this warp has read back to the copies that fill them. (The
// fence is needed: an arrival alone is performed while loads are on their way, and without it the
// next part's bytes were unpacked in the place of this one's.)
__device__ __forceinline__ void give_back(uint64_t *bar, int lane) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}

// A chunk's row of a key in shared memory without its infinities and NaN.
static __device__ __noinline__ void make_finite(uint32_t row) {
#pragma unroll 1
    for (int w = 0; w < 8; ++w) {
        uint32_t v[4];
        load_piece(v, row ^ (16 * w));
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = finite2(v[j]);
        store_piece(row ^ (16 * w), v);
    }
}

// A key's 64 dims from TMEM to its row in shared memory, without infinities and NaN.
__device__ __forceinline__ void copy_chunk(uint32_t col, uint32_t to, bool odd) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint32_t v[16];
        tmem_ld16(col + 16 * k, v);
        tmem_wait_ld();
#pragma unroll
        for (int w = 0; w < 4; ++w) store_piece(to ^ (64 * k + 16 * w), v + 4 * w);
    }
    if (odd) make_finite(to);
    fence_proxy_async_smem();
}

// The softmax warps form two groups of four, one per half of the rows (named barriers 1 and
// 2, 128 threads each).
__device__ __forceinline__ bool vote_any_group(bool pred, int hh) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n bar.red.or.pred q, %2, 128, p;\n"
        " selp.b32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(pred)), "r"(1 + hh)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ void bar_group(int hh) {
    asm volatile("bar.sync %0, 128;" ::"r"(1 + hh) : "memory");
}

// Products that a row of q must not see become -inf.
__device__ __forceinline__ void hide32(uint32_t (&s)[32], uint32_t vis) {
#pragma unroll
    for (int j = 0; j < 32; ++j)
        if (!((vis >> j) & 1u)) s[j] = __float_as_uint(-INFINITY);
}

// The largest of the 32 products less their rows' running maxima (which are negated).
__device__ __forceinline__ float over_max(const uint32_t (&s)[32], const float *minus_m) {
    const ulonglong2 *m2 = reinterpret_cast<const ulonglong2 *>(minus_m);
    float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const ulonglong2 m = m2[j];
        const uint64_t a = add_pair(pair_of(s[4 * j], s[4 * j + 1]), m.x);
        const uint64_t b = add_pair(pair_of(s[4 * j + 2], s[4 * j + 3]), m.y);
        t[j & 1] = max3(t[j & 1], first_of(a), second_of(a));
        t[2 + (j & 1)] = max3(t[2 + (j & 1)], first_of(b), second_of(b));
    }
    return max3(fmaxf(t[0], t[1]), t[2], t[3]);
}

// ------------------------------------------------------------------ the kernel

__global__ void __launch_bounds__(kT, 1)
    q4_attn_kernel(const __grid_constant__ CUtensorMap tm_q,
                   const __grid_constant__ CUtensorMap tm_raw,
                   const __grid_constant__ CUtensorMap tm_rope,
                   const __grid_constant__ SinkParams p, const uint8_t *pages) {
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *sQ = smem + kOffQ;
    uint8_t *sV = smem + kOffV;
    uint8_t *s6 = smem + kOff6;
    uint8_t *sP = smem + kOffP;
    float *sRed = reinterpret_cast<float *>(smem + kOffRed);
    float *sL = sRed;
    float *sLinv = reinterpret_cast<float *>(smem + kOffLinv);
    float *sAlpha = sLinv;
    float *sM = reinterpret_cast<float *>(smem + kOffM);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kOffBar);
    uint64_t *tm_full = bars + 0;   // [3] pair of chunks 0-5 in TMEM
    uint64_t *v_full = bars + 3;    // [3] pair of chunks 0-5 in shared memory
    uint64_t *v_free = bars + 6;    // [4] pair of chunks used by PV
    uint64_t *k6_full = bars + 10;  // chunk 6 unpacked
    uint64_t *raw_free = bars + 11; // [4] a part of the 4-bit bytes taken
    uint64_t *raw_full = bars + 15; // [4] ... landed
    uint64_t *r_full = bars + 19;   // chunk 7 landed
    uint64_t *qa_done = bars + 20;  // QK has read the chunks in TMEM
    uint64_t *q_full = bars + 21;
    uint64_t *q_free = bars + 22;
    uint64_t *q_turned = bars + 23;
    uint64_t *s_full = bars + 24;
    uint64_t *s_free = bars + 25;
    uint64_t *p_full = bars + 26;
    uint64_t *pv_done = bars + 27;  // P may be written, O rescaled
    uint64_t *o_full = bars + 28;
    uint64_t *o_free = bars + 29;
    uint64_t *drain = bars + 30;    // [2] one per issuing warp
    constexpr int kBars = 32;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + kBars);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    int *sStart = reinterpret_cast<int *>(tmem_holder + 2);    // [5] start of this CTA's run
    volatile uint32_t *sBlocks = tmem_holder + 1 + kBlocksAt;  // blocks begun
    volatile uint32_t *sMore = tmem_holder + 10;               // [kRing] 0: the run has ended
    volatile uint32_t *sValid = sMore + kRing;                 // [kRing][4] keys that are there

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (smem_u32(smem) & 1023u) {  // the tiles' swizzle counts on it
        wait_before();
        if (tid == 0) {
            report(p.status, DSA_ERR_CUDA);
            reinterpret_cast<JoinDesc *>(p.ws + kWsDesc)[blockIdx.x] = JoinDesc{};
        }
        return;
    }
    if (warp == 0) {
        // arrivals a phase takes: 8 unpacking warps on tm_full, v_full, k6_full and raw_free, the
        // turning warp's threads on q_turned, 8 softmax warps on s_free, p_full and o_free, one on
        // the others
        int n = 1;
        uint64_t *bar = bars + lane;
        if (bar < v_free || (bar >= k6_full && bar < raw_full)) n = 8;
        if (bar == q_turned) n = 32;
        if (bar == s_free || bar == o_free || bar == p_full) n = 8;
        mbar_init(bar, n);
        if (lane == 31) {
            *abort_flag = 0;
            sStart[4] = 0;
            *sBlocks = 0;
        }
        fence_barrier_init();
    }
    if (warp == kPvWarp) tmem_alloc(tmem_holder, 512);
    if (tid == 32 * kQWarp) {
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_raw);
        prefetch_tmap(&tm_rope);
    }
    wait_before();
    const int cta = static_cast<int>(blockIdx.x);
    find_run<kT>(p, reinterpret_cast<int64_t *>(sV), sStart);
    // All 512 columns of TMEM begin at 0: known addresses, which the products take without a move.
    constexpr uint32_t tmem = 0;
    if (tid == 0 && *tmem_holder != tmem) {
        *abort_flag = 1;
        report(p.status, DSA_ERR_CUDA);
    }

    if (warp < kUnpackWarp0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLow));
        if (warp == 0) {
            // ---------------- the 4-bit bytes, 64 of a row at a time. Lane i < np loads page i;
            // a block's table entries are read, and its rows brought to L2, one block ahead.
            const int prows = min(1 << p.b.page_shift, kBlock), np = kBlock / prows;
            const int key_shift = min(p.b.page_shift, 7);
            const uint64_t once = policy_evict_first(), keep = policy_evict_normal();
            PageWalk walk(p, sStart);
            bool have = false, have_next, ok = true;
            int32_t e = -1, e_next = -1;
            int row = 0, row_next = 0;
            // keys [a, b) and those below c of a block are seen by some token
            int a = 0, b = 0, c = 0, a_next = 0, b_next = 0, c_next = 0;
            bool alone = false, alone_next = false;
            int parts = 0;   // loaded so far
            for (int t = -1;; ++t) {
                have_next = walk.have;
                if (have_next) {
                    const int pos = walk.x.block_pos(walk.b);
                    a_next = walk.x.lo - pos;
                    b_next = walk.x.posl - pos + 1;
                    c_next = walk.b == 0 && walk.x.ahead > 0 ? p.sinks : p.sinks - pos;
                    alone_next = walk.x.alone;
                    e_next = walk.next(p, lane, prows, np, row_next);
                    if (e_next >= 0)
                        prefetch_rows(pages + e_next * p.b.page_stride + int64_t{row_next} * kQ4Row,
                                      prows * kQ4Row);
                }
                if (t >= 0) {
                    *sBlocks = static_cast<uint32_t>(t) + 1;
                    const uint32_t mask = __ballot_sync(0xFFFFFFFFu, e >= 0);
                    const uint32_t bytes = static_cast<uint32_t>(__popc(mask)) * prows * 64;
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const int key = 32 * w + lane;
                        const uint32_t there = __ballot_sync(
                            0xFFFFFFFFu, ((mask >> (key >> key_shift)) & 1u) && key < b &&
                                             (key >= a || key < c));
                        if (lane == w) sValid[4 * (t & (kRing - 1)) + w] = there;
                    }
                    if (lane == 4) sMore[t & (kRing - 1)] = have;
                    __syncwarp();
#pragma unroll 1
                    for (int j = 0; j < 4; ++j) {
                        // (the part before in the slot: 2, 3 of the last block, then 0, 1)
                        ok = __all_sync(0xFFFFFFFFu,
                                        wait_bar(&raw_free[j ^ 2], (t & 1) ^ (j < 2), abort_flag,
                                                 p.status));
                        if (!ok) break;
                        if (!have) {
                            if (lane == 0) mbar_arrive(&raw_full[0]);
                            break;
                        }
                        ++parts;
                        if (lane == 0) mbar_expect_tx(&raw_full[j], bytes);
                        __syncwarp();
                        if (e >= 0)
                            tma_load_3d(smem + kOffRaw + (j & 1) * 8192 + lane * prows * 64,
                                        &tm_raw, &raw_full[j], 32 * j, row, e,
                                        alone ? once : keep);
                    }
                    if (!ok || !have) break;
                }
                have = have_next;
                e = have_next ? e_next : -1;
                row = row_next;
                a = a_next;
                b = b_next;
                c = c_next;
                alone = alone_next;
            }
            // no copy into this CTA's shared memory may still be in flight at exit
            __syncwarp();
            if (lane == 0) {
                for (int l = max(0, parts - 2); l < parts; ++l)
                    drain_wait(&raw_full[l & 3], (l >> 2) & 1);
            }
            __syncwarp();
        } else if (warp == kQkWarp) {
            // ---------------- QK. (It and PV are issued by a warp each, so that neither waits for
            // what the other one needs.)
            constexpr uint32_t idesc_qk = idesc_bf16(kBlock, kRows, false, false);
            const bool turn = p.b.cos_sin && p.turn_q;
            Walk walk(p, sStart);
            Segment x;
            int i = 0, g = 0;
            bool ok = true;
            for (; ok && walk.next(p, x); ++i) {
                if (!(ok = wait_bar(q_full, i & 1, abort_flag, p.status))) break;
                for (int b = 0; b < x.nb; ++b, ++g) {
                    if (!(ok = wait_bar(s_free, (g & 1) ^ 1, abort_flag, p.status))) break;
#pragma unroll 1
                    for (int m = 0; m < 3; ++m) {   // chunks 0-5
                        if (!(ok = wait_bar(&tm_full[m], g & 1, abort_flag, p.status))) break;
                        tc_fence_after();
                        if (elect_one()) {
                            const uint64_t bd = desc_sw128(smem_u32(sQ) + 2 * m * 8192, 16, 1024);
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                mma_bf16_ta(tmem + kSCol, tmem + kKCol + 64 * m + 8 * k,
                                            bd + (k / 4) * (8192 >> 4) + 2 * (k % 4), idesc_qk,
                                            m > 0 || k > 0);
                            if (m == 2) mma_commit(qa_done);
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                    // chunk 6 and chunk 7
                    if (!(ok = wait_bar(k6_full, g & 1, abort_flag, p.status))) break;
                    if (!(ok = wait_bar(r_full, g & 1, abort_flag, p.status))) break;
                    if (b == 0 && turn && !(ok = wait_bar(q_turned, i & 1, abort_flag, p.status)))
                        break;
                    tc_fence_after();
                    if (elect_one()) {
                        const uint64_t bd = desc_sw128(smem_u32(sQ) + 6 * 8192, 16, 1024);
                        const uint64_t a6 = desc_sw128(smem_u32(s6), 16, 1024);
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            mma_bf16(tmem + kSCol, a6 + (k / 4) * (kChunk >> 4) + 2 * (k % 4),
                                     bd + (k / 4) * (8192 >> 4) + 2 * (k % 4), idesc_qk, 1u);
                        mma_commit(s_full);
                        if (b == x.nb - 1) mma_commit(q_free);
                    }
                    __syncwarp();
                }
            }
            if (elect_one()) {
                mma_commit(&drain[0]);
                drain_wait(&drain[0], 0);
            }
            __syncwarp();
        } else if (warp == kPvWarp) {
            // ---------------- PV, tile by tile: the last one first, as its chunk 6 is what QK of
            // the next block waits for
            constexpr uint32_t idesc_pv = idesc_bf16(128, kRows, true, true);
            Walk walk(p, sStart);
            Segment x;
            int i = 0, g = 0;
            bool ok = true;
            for (; ok && walk.next(p, x); ++i) {
                for (int b = 0; b < x.nb && ok; ++b, ++g) {
                    if (!(ok = wait_bar(p_full, g & 1, abort_flag, p.status))) break;
                    // the results of the unit before must have left O^T
                    if (b == 0 && i > 0 &&
                        !(ok = wait_bar(o_free, (i - 1) & 1, abort_flag, p.status)))
                        break;
#pragma unroll 1
                    for (int st = 0; st < 4; ++st) {
                        const int m = (st + 3) & 3;   // dims 128 m ..
                        if (st > 0 && !(ok = wait_bar(&v_full[m], g & 1, abort_flag, p.status)))
                            break;
                        tc_fence_after();
                        if (elect_one()) {
                            const uint64_t ad = desc_sw128(
                                smem_u32(smem) + (st > 0 ? kOffV + 2 * m * kChunk : kOff6),
                                kChunk, 1024);
                            const uint64_t bd = desc_sw128(smem_u32(sP), 8192, 1024);
#pragma unroll
                            for (int kk = 0; kk < 8; ++kk)
                                mma_bf16(tmem + kOCol + 64 * m, ad + ((kk * 2048) >> 4),
                                         bd + ((kk * 2048) >> 4), idesc_pv, kk > 0 || b > 0);
                            mma_commit(&v_free[m]);
                            if (st == 3) {
                                mma_commit(pv_done);
                                if (b == x.nb - 1) mma_commit(o_full);
                            }
                        }
                        __syncwarp();
                    }
                }
            }
            if (elect_one()) {
                mma_commit(&drain[1]);
                drain_wait(&drain[1], 0);
            }
            __syncwarp();
        } else {
            // ---------------- the queries, loaded when the last unit's products have read theirs and
            // turned in place, two rows a thread; and chunk 7 of each block, when PV of the block
            // before has used it
            const bool turn = p.b.cos_sin && p.turn_q;
            const int prows = min(1 << p.b.page_shift, kBlock), np = kBlock / prows;
            const uint64_t once = policy_evict_first(), keep = policy_evict_normal();
            Walk walk(p, sStart);
            Segment x;
            int i = 0, t = 0;
            bool ok = true;
            for (; ok && walk.next(p, x); ++i) {
                if (!(ok = __all_sync(0xFFFFFFFFu,
                                      wait_bar(q_free, (i & 1) ^ 1, abort_flag, p.status))))
                    break;
                if (lane == 0) {
                    mbar_expect_tx(q_full, 65536);
                    for (int c = 0; c < 8; ++c)
                        tma_load_2d(sQ + c * 8192, &tm_q, q_full, c * 64, static_cast<int>(x.row),
                                    once);
                }
                __syncwarp();
                for (int b = 0; b < x.nb; ++b, ++t) {
                    // (a bad table entry is reported by the other loader)
                    const int pos = x.key_pos(b, lane * prows);
                    int32_t e = -1;
                    if (lane < np && pos <= x.posl && (pos > x.lo - prows || pos < p.sinks))
                        e = __ldg(p.b.page_table + int64_t{x.s} * p.b.max_pages +
                                  (pos >> p.b.page_shift));
                    const bool there = e >= 0 && e < p.b.n_pages;
                    const uint32_t mask = __ballot_sync(0xFFFFFFFFu, there);
                    if (!(ok = __all_sync(0xFFFFFFFFu,
                                          t == 0 || wait_bar(&v_free[3], (t - 1) & 1, abort_flag,
                                                             p.status))))
                        break;
                    if (lane == 0)
                        mbar_expect_tx(r_full, static_cast<uint32_t>(__popc(mask)) * prows * 128);
                    __syncwarp();
                    if (there)
                        tma_load_3d(smem + kOff7 + lane * prows * 128, &tm_rope, r_full,
                                    kQ4Rope / 2, pos & ((1 << p.b.page_shift) - 1), e,
                                    x.alone ? once : keep);
                    if (b > 0 || !turn) continue;
                    if (!(ok = __all_sync(0xFFFFFFFFu,
                                          wait_bar(q_full, i & 1, abort_flag, p.status)))) {
                        ++t;
                        break;
                    }
#pragma unroll 1
                    for (int r = lane; r < x.nrows; r += 32) {
                        uint8_t *row = sQ + 7 * 8192 + r * 128;
                        const float4 *src = reinterpret_cast<const float4 *>(
                            p.b.cos_sin + int64_t{row_pos(p, x.posf, r)} * kRope);
#pragma unroll 4
                        for (int k = 0; k < 8; ++k) {
                            const float4 c0 = __ldg(src + 2 * k), c1 = __ldg(src + 2 * k + 1);
                            uint4 *at = reinterpret_cast<uint4 *>(row + ((k ^ (r & 7)) << 4));
                            uint4 v = *at;
                            v.x = turn_pair(v.x, c0.x, c0.y);
                            v.y = turn_pair(v.y, c0.z, c0.w);
                            v.z = turn_pair(v.z, c1.x, c1.y);
                            v.w = turn_pair(v.w, c1.z, c1.w);
                            *at = v;
                        }
                    }
                    fence_proxy_async_smem();
                    mbar_arrive(q_turned);
                }
                if (!ok) {
                    ++i;
                    break;
                }
            }
            // no copy into this CTA's shared memory may still be in flight at exit
            if (lane == 0) {
                if (i > 0) drain_wait(q_full, (i - 1) & 1);
                if (t > 0) drain_wait(r_full, (t - 1) & 1);
            }
            __syncwarp();
        }
    } else if (warp < kSoftWarp0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLow));
        // ---------------- unpacking. Step t: chunk 6 of block t - 1 (a half by each half of the
        // warps), then pair by pair the bytes of block t into registers, the chunks of block t - 1
        // from TMEM to shared memory and those of block t into TMEM. (Once the kernel gives up no
        // wait lasts, and the next block does not come.)
        const int sp = warp & 3, h = (warp - kUnpackWarp0) >> 2;
        const int key = 32 * sp + lane;
        const uint32_t k_col = tmem + (static_cast<uint32_t>(sp * 32) << 16) + kKCol + 32 * h;
        // (piece w of a swizzled row lies at the row's place ^ 16 w)
        const uint32_t row_at = key * 128 + ((key & 7) << 4);
        const uint32_t to6 = (smem_u32(s6) + row_at) ^ (64 * h);
        const uint32_t to_v = smem_u32(sV) + h * kChunk + row_at;
        const uint32_t from = smem_u32(smem) + kOffRaw + key * 64 + (((key >> 1) & 3) << 4);

        uint32_t raw6[4], two[3], two6 = 0;  // bytes of chunk 6's half; scales of the chunks' halves
        float pow = 0.0f;                    // half of the row's power of two
        bool odd = false;                    // a scale that is NaN, in the block to be copied
        bool have = true, before = false;    // block t is there, block t - 1 is to be copied
        for (int t = 0;; ++t) {
            if (before) {
                // chunk 6 of block t - 1, in the place that PV of block t - 2 has left
                uint32_t v[16];
                unpack32(raw6, two6 & 0xFFFFu, pow, v);
                if (t > 1) wait_bar(&v_free[3], t & 1, abort_flag, p.status);
#pragma unroll
                for (int w = 0; w < 4; ++w) store_piece(to6 ^ (16 * w), v + 4 * w);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(k6_full);
            }
            bool odd_next = false;
            if (have) {
                const bool ok =
                    __all_sync(0xFFFFFFFFu, wait_bar(&raw_full[0], t & 1, abort_flag, p.status));
                have = ok && sMore[t & (kRing - 1)];
            }
            if (!have && !before) break;
            if (have) {
                // the scales (of a key that is not there: zeros, and so are its values)
                uint32_t head[8];
                load_piece(head, from);
                load_piece(head + 4, from ^ 16);
                const bool there = (sValid[4 * (t & (kRing - 1)) + sp] >> lane) & 1u;
#pragma unroll
                for (int m = 0; m < 3; ++m)   // chunk 2 m + h: bytes 4 m + 2 h of either half
                    two[m] = there ? __byte_perm(head[m], head[4 + m], h ? 0x7632 : 0x5410) : 0u;
                two6 = there ? (h ? head[7] : head[3]) : 0u;  // chunk 6, half h: bytes 12 and 13
                odd_next = has_nan(two[0]) || has_nan(two[1]) || has_nan(two[2]);
                pow = pow2(q4_exp((head[3] >> 16) & 0xFFu) - 1);
                if (h == 1) give_back(&raw_free[0], lane);
            }
            // (one copy of the code for the three pairs: fetching it costs more than the loop)
#pragma unroll 1
            for (int m = 0; m < 3; ++m) {
                uint32_t raw[8];
                const int part = m + h;
                if (have) {
                    // the 32 bytes of chunk 2 m + h: half (1 - h) of part m + h (before the copy:
                    // the next part is on its way the earlier; 5.09 -> 4.70 ms for 2,048 tokens at
                    // 16,384)
                    const uint32_t at = (from + (part & 1) * 8192) ^ (h ? 0 : 32);
                    wait_bar(&raw_full[part], t & 1, abort_flag, p.status);
                    load_piece(raw, at);
                    load_piece(raw + 4, at ^ 16);
                    if (part < 3) give_back(&raw_free[part], lane);
                }
                if (before) {
                    if (t > 1) wait_bar(&v_free[m], t & 1, abort_flag, p.status);
                    copy_chunk(k_col + 64 * m, to_v + 2 * m * kChunk, odd);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&v_full[m]);
                    if (m == 0 && have) {    // QK of block t - 1 has read what is overwritten
                        wait_bar(qa_done, (t - 1) & 1, abort_flag, p.status);
                        tc_fence_after();
                    }
                }
                if (have) {
                    if (m == 2) {
                        // and those of chunk 6: the second half of part 3
                        if (h == 0) wait_bar(&raw_full[3], t & 1, abort_flag, p.status);
                        load_piece(raw6, (from + 8192) ^ (32 + 16 * h));
                        give_back(&raw_free[3], lane);
                    }
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t v[16];
                        unpack32(raw + 4 * half, (two[0] >> (16 * half)) & 0xFFFFu, pow, v);
                        tmem_st16(k_col + 64 * m + 16 * half, v);
                    }
                    two[0] = two[1];
                    two[1] = two[2];
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&tm_full[m]);
                }
            }
            odd = odd_next;
            before = have;
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
        // ---------------- softmax + epilogue, 8 warps: TMEM lanes of sub-partition sp (keys,
        // later dims) x rows [32 hh, 32 hh + 32)
        const int sp = warp & 3;
        const int hh = (warp - kSoftWarp0) >> 2;
        const int hb = 32 * hh;
        const int kl = sp * 32 + lane;
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(sp * 32) << 16);
        // (the walk and the segments in shared memory, the half's own: registers are few)
        SoftWalk &mine = reinterpret_cast<SoftWalk *>(smem + kOffWalk)[hh];
        auto step_walk = [&](int at) {
            Walk w = mine.walk;
            Segment next;
            mine.more[at] = w.next(p, next);
            mine.x[at] = next;
            mine.walk = w;
        };
        if (sp == 0 && lane == 0) {
            mine.walk = Walk(p, sStart);
            step_walk(0);
        }
        bar_group(hh);
        int i = 0, g = 0, cur = 0;
        for (;; ++i) {
            const Segment &x = mine.x[i & 1];
            if (!mine.more[i & 1]) break;
            uint64_t l[16];   // sums of rows 2 j and 2 j + 1, over this lane's keys
#pragma unroll
            for (int j = 0; j < 16; ++j) l[j] = 0;
            if (sp == 0) sM[cur * 64 + hb + lane] = -kNoMax;
            bar_group(hh);
            // (the next segment, while the first products are on their way; in the place of the one
            // before, which the whole group has left)
            if (sp == 0 && lane == 0) step_walk((i + 1) & 1);
            for (int b = 0; b < x.nb; ++b, ++g) {
                const int k0 = x.block_pos(b);
                const bool live = __all_sync(
                    0xFFFFFFFFu, mbar_wait(s_full, g & 1, abort_flag, p.status));
                // (complete since QK of this block waited for it: orders sValid before here)
                mbar_wait(k6_full, g & 1, abort_flag, p.status);
                tc_fence_after();
                const uint32_t s_col = lane_base + kSCol + hb;
                uint32_t sa[32];
                const uint32_t valid = sValid[4 * (g & (kRing - 1)) + sp];
                if (live) tmem_ld32(s_col, sa);
                // every row sees every key of the warp, unless ...
                const bool masked = k0 + 32 * sp + 31 > x.posf ||
                                    (p.window > 0 && k0 <= x.posl - p.window) ||
                                    valid != 0xFFFFFFFFu || !live;
                tmem_wait_ld();
                // S may take QK of the next block
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_free);
                if (masked) {
                    // rows [ra, rb) of the unit see the key: their token is not before it and
                    // less than `window` after it, or it is one of the first
                    const int pos = x.key_pos(b, kl);
                    const int64_t ahead = int64_t{pos} - x.posf;
                    const int ta = static_cast<int>(max(int64_t{0}, min(ahead, int64_t{64})));
                    const int64_t gone =
                        p.window > 0 && pos >= p.sinks ? ahead + p.window : 64;
                    const int tb = static_cast<int>(max(int64_t{0}, min(gone, int64_t{64})));
                    const int ra = min(64, ta * p.rpt);
                    int rb = min(64, tb * p.rpt);
                    if (!((valid >> lane) & 1u) || !live) rb = 0;
                    const int a = max(0, min(32, ra - hb)), e = max(0, min(32, rb - hb));
                    const uint32_t below_e = e == 32 ? 0xFFFFFFFFu : (1u << e) - 1u;
                    const uint32_t below_a = a == 32 ? 0xFFFFFFFFu : (1u << a) - 1u;
                    const uint32_t vis = below_e & ~below_a;   // rows hb + j that see the key
                    // A row of the cache that holds an infinity or NaN makes its logit non-finite
                    // in every row of q. Where a row of q must not see the key, those elements
                    // become zero in the tile (0 * inf in PV would reach every row); rows that
                    // do see the key have a NaN probability already, or with a logit of -inf
                    // give it no weight. Chunks 0-5 are finite in shared memory; the others a key
                    // at a time: lane = 16-byte piece of the two.
                    uint64_t t2[2] = {0, 0};  // NaN if any is not finite
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        t2[j & 1] = fma_pair(pair_of(sa[2 * j], sa[2 * j + 1]), 0, t2[j & 1]);
                    t2[0] = add_pair(t2[0], t2[1]);
                    const bool odd = !(first_of(t2[0]) + second_of(t2[0]) == 0.0f);
                    hide32(sa, vis);
                    uint32_t keys =
                        __ballot_sync(0xFFFFFFFFu, odd && live && (ra > 0 || rb < x.nrows));
                    if (keys) {
                        mbar_wait(r_full, g & 1, abort_flag, p.status);
                        uint8_t *tile = s6 + (lane >> 3) * kChunk + sp * 4096 + (lane & 7) * 16;
#pragma unroll 1
                        for (; keys && lane < 16; keys &= keys - 1) {
                            uint4 *at = reinterpret_cast<uint4 *>(tile + (__ffs(keys) - 1) * 128);
                            uint4 v = *at;
                            v.x = finite2(v.x);
                            v.y = finite2(v.y);
                            v.z = finite2(v.z);
                            v.w = finite2(v.w);
                            *at = v;
                        }
                        __syncwarp();
                    }
                }
                if (vote_any_group(over_max(sa, sM + cur * 64 + hb) * p.c > kRescale, hh)) {
                    // exact block maxima -> new running maximum; sums and O^T rescaled
                    // (transposed and reduced over the warp's keys as the sums below: lane = row; a
                    // redux.sync per row takes 4,000 cycles here, with all eight warps at it)
                    float top[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const bool up = (lane & 16) != 0;
                        const float lo = __uint_as_float(sa[j]), hi = __uint_as_float(sa[j + 16]);
                        top[j] = fmaxf(up ? hi : lo,
                                       __shfl_xor_sync(0xFFFFFFFFu, up ? lo : hi, 16));
                    }
#pragma unroll
                    for (int w = 8; w >= 1; w >>= 1) {
                        const bool up = (lane & w) != 0;
#pragma unroll
                        for (int j = 0; j < w; ++j)
                            top[j] = fmaxf(up ? top[j + w] : top[j],
                                           __shfl_xor_sync(0xFFFFFFFFu, up ? top[j] : top[j + w], w));
                    }
                    sRed[sp * 64 + hb + lane] = top[0];
                    bar_group(hh);
                    if (sp == 0) {
                        const int r = hb + lane;
                        const float bm = fmaxf(fmaxf(sRed[r], sRed[64 + r]),
                                               fmaxf(sRed[128 + r], sRed[192 + r]));
                        const float m_old = -sM[cur * 64 + r];
                        const float m_new = fmaxf(m_old, bm);
                        sM[(cur ^ 1) * 64 + r] = -m_new;
                        sAlpha[r] = ex2((m_old - m_new) * p.c);
                    }
                    bar_group(hh);
                    cur ^= 1;
                    const uint64_t *alpha = reinterpret_cast<const uint64_t *>(sAlpha + hb);
#pragma unroll
                    for (int j = 0; j < 16; ++j) l[j] = mul_pair(l[j], alpha[j]);
                    if (b > 0 && live) {
                        mbar_wait(pv_done, (g & 1) ^ 1, abort_flag, p.status);
                        tc_fence_after();
#pragma unroll 1
                        for (int m = 0; m < 16; ++m) {
                            uint32_t oa[8];
                            const uint32_t col = lane_base + kOCol + 64 * (m / 4) + hb + 8 * (m & 3);
                            tmem_ld8(col, oa);
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                oa[j] = __float_as_uint(__uint_as_float(oa[j]) *
                                                        sAlpha[hb + 8 * (m & 3) + j]);
                            tmem_st8(col, oa);
                        }
                        tmem_wait_st();
                    }
                }
                // this thread's 32 rows of P^T for key kl. The sums take P as rounded to bf16, the
                // values that PV multiplies.
                uint32_t pk[16];
                const uint64_t c2 = pair_of(p.c);
                const uint64_t *m2 = reinterpret_cast<const uint64_t *>(sM + cur * 64 + hb);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const uint64_t y =
                        mul_pair(add_pair(pair_of(sa[2 * j], sa[2 * j + 1]), m2[j]), c2);
                    const __nv_bfloat162 v =
                        __floats2bfloat162_rn(ex2(first_of(y)), ex2(second_of(y)));
                    pk[j] = *reinterpret_cast<const uint32_t *>(&v);
                    l[j] = add_pair(l[j], pair_of(pk[j] << 16, pk[j] & 0xFFFF0000u));
                }
                // PV of the block before has used P
                mbar_wait(pv_done, (g & 1) ^ 1, abort_flag, p.status);
                {
                    uint8_t *prow = sP + kl * 128;
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        *reinterpret_cast<uint4 *>(prow + (((4 * hh + q) ^ (kl & 7)) << 4)) =
                            make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]);
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full);
            }
            // ---- end of the segment: sums over the keys. Transpose-reduce the 32 partial
            // sums across the warp: lane ends with the warp's total for row hb + lane
            float lf[32];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                lf[2 * j] = first_of(l[j]);
                lf[2 * j + 1] = second_of(l[j]);
            }
#pragma unroll
            for (int w = 16; w >= 1; w >>= 1) {
                const bool up = (lane & w) != 0;
#pragma unroll
                for (int j = 0; j < w; ++j) {
                    const float send = up ? lf[j] : lf[j + w];
                    const float keep = up ? lf[j + w] : lf[j];
                    lf[j] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, w);
                }
            }
            sL[sp * 64 + hb + lane] = lf[0];
            bar_group(hh);
            const int slot = 2 * cta + (i > 0);
            if (sp == 0) {
                // (each half's own warp: `cur` goes by the half)
                const int r = hb + lane;
                const float tot = sL[r] + sL[64 + r] + sL[128 + r] + sL[192 + r];
                // a row that saw no key has sum 0 and O 0
                sLinv[r] = tot == 0.0f ? 0.0f : 1.0f / tot;
                if (!x.whole)
                    reinterpret_cast<float2 *>(p.ws + kWsMl)[slot * kMaxRows + r] =
                        make_float2(-sM[cur * 64 + r], tot);
            }
            bar_group(hh);
            // O^T into registers one d-tile at a time: lane holds dim 128 m + 32 sp + lane of
            // rows hb .. hb + 31, so a warp writes 32 consecutive dims of each row
            // (8 rows a step: the code stays where it is fetched from, and is fetched once)
            const int rows = min(32, x.nrows - hb);
            const uint32_t o_col = lane_base + kOCol + hb;
            if (x.whole) {
                __nv_bfloat16 *o = p.out + (x.row + hb) * kD + 32 * sp + lane;
                // turned back by the token's position; a pair is in two adjacent lanes
                const bool turns = p.b.cos_sin && sp >= 2;
                const float2 *cs =
                    reinterpret_cast<const float2 *>(p.b.cos_sin) + ((sp - 2) * 16 + (lane >> 1));
                // (a unit of one token's heads has one position)
                int pos = p.tpu == 1 ? x.posf : x.posf + hb / p.rpt;
                int left = p.tpu == 1 ? kRows : p.rpt - hb % p.rpt;  // rows at pos
                const bool live = mbar_wait(o_full, i & 1, abort_flag, p.status);
                tc_fence_after();
#pragma unroll 1
                for (int m = 0; m < 16; ++m) {    // dims 128 (m / 4) .., rows 8 (m % 4) ..
                    uint32_t oa[8];
                    if (!__all_sync(0xFFFFFFFFu, live)) break;
                    const int j0 = 8 * (m % 4);
                    tmem_ld8(o_col + 64 * (m / 4) + j0, oa);
                    tmem_wait_ld();
                    __nv_bfloat16 *to = o + 128 * (m / 4) + j0 * kD;
                    const float *inv = sLinv + hb + j0;
                    if (turns && m >= 12) {
                        float2 a[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            a[j] = __ldg(cs + int64_t{min(pos, x.posl)} * kRopePairs);
                            const bool last = --left == 0;
                            pos += last;
                            left = last ? p.rpt : left;
                        }
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float v = __uint_as_float(oa[j]) * inv[j];
                            const float w = __shfl_xor_sync(0xFFFFFFFFu, v, 1);
                            if (j0 + j < rows)
                                to[j * kD] =
                                    __float2bfloat16_rn(v * a[j].x + (lane & 1 ? -w : w) * a[j].y);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (j0 + j < rows)
                                to[j * kD] = __float2bfloat16_rn(__uint_as_float(oa[j]) * inv[j]);
                    }
                }
            } else {
                float *o = reinterpret_cast<float *>(p.ws + kWsO) +
                           (int64_t{slot} * kRows + hb) * kD + 32 * sp + lane;
                const bool live = mbar_wait(o_full, i & 1, abort_flag, p.status);
                tc_fence_after();
#pragma unroll 1
                for (int m = 0; m < 16; ++m) {
                    uint32_t oa[8];
                    if (!__all_sync(0xFFFFFFFFu, live)) break;
                    const int j0 = 8 * (m % 4);
                    tmem_ld8(o_col + 64 * (m / 4) + j0, oa);
                    tmem_wait_ld();
                    float *to = o + 128 * (m / 4) + j0 * kD;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (j0 + j < rows) to[j * kD] = __uint_as_float(oa[j]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_free);
        }
    }
    __syncthreads();
    if (warp == kPvWarp) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------ host

std::mutex g_mu;
int g_sms[kMaxDevices];   // 0: not set up yet

// Per-device one-time set-up. A failure is not kept: it may pass (memory for the module's code).
int setup(int *sms) {
    const int dev = current_device();
    if (dev < 0) return DSA_ERR_CUDA;
    std::lock_guard<std::mutex> lock(g_mu);
    if (!g_sms[dev]) {
        const int n = sm_count();
        const int rc = n > 0 ? prepare_kernel(q4_attn_kernel, kRegsLaunch, kSmem) : DSA_ERR_CUDA;
        if (rc != DSA_OK) return rc;
        g_sms[dev] = n;
    }
    *sms = g_sms[dev];
    return DSA_OK;
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
    SinkParams p;
    int rc = check_paged_batch(n_new, new_start, seq_len, n_seqs, page_table, max_pages, pages,
                               n_pages, page_stride, page_size, cos_sin, n_pos, &p.b, kQ4PageRow);
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
    p.heads = heads;
    p.rows = kRows;
    p.tpu = heads <= kRows ? kRows / heads : 1;
    p.upt = (heads + kRows - 1) / kRows;
    p.row_step = kRows;
    p.rpt = std::min(heads, p.rows);
    // a window no shorter than any sequence is no window
    p.window = window >= p.b.len_limit ? 0 : window;
    p.sinks = p.window > 0 ? sinks : 0;
    const int prows = std::min(page_size, kBlock);
    p.sink_keys = (p.sinks + prows - 1) / prows * prows;
    p.turn_q = !q_turned;
    const int64_t keys =
        p.window > 0 ? std::min(p.b.len_limit, p.window + p.tpu) + kBlock : p.b.len_limit;
    if (paged_run_bound(p, keys) > (int64_t{1} << 31) - 1) return DSA_ERR_SHAPE;
    if (!workspace || !aligned16(workspace) || workspace_bytes < used) return DSA_ERR_SCRATCH;
    if (overlaps(workspace, used, q, bytes) || overlaps(workspace, used, out, bytes) ||
        touches_pages(p.b, pages, workspace, used, kQ4PageRow))
        return DSA_ERR_ARG;
    p.out = static_cast<__nv_bfloat16 *>(out);
    // whole lines (the caller's buffer begins on 16 bytes at least)
    p.ws = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(workspace) + (kWsAlign - 1)) &
                                       ~uintptr_t{kWsAlign - 1});
    p.c = c;
    p.status = dev_status;
    int sms = 0;
    rc = setup(&sms);
    if (rc != DSA_OK) return rc;
    CUtensorMap tm_q, tm_raw, tm_rope;
    if (!make_tmap_bf16(&tm_q, q, kD, static_cast<uint64_t>(n_new) * heads, kD * 2, 64, p.rows) ||
        !make_tmap_pages(&tm_raw, pages, p.b, kQ4PageRow, 32) ||
        !make_tmap_pages(&tm_rope, pages, p.b, kQ4PageRow))
        return DSA_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int ctas = std::min(sms, kMaxCtas);
    rc = launch_overlapped(q4_attn_kernel, ctas, kT, kSmem, s, tm_q, tm_raw, tm_rope, p,
                           static_cast<const uint8_t *>(pages));
    return rc == DSA_OK ? enqueue_paged_join(p, ctas, s) : rc;
}
