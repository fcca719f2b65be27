// dsa_paged_attn for chunks: units of up to 128 rows of q (whole tokens of one sequence) and half
// of the output dims.
//
// The kernel for few rows (paged_attn.cu) keeps one 128-key tile of all 512 dims beside 64
// rows of q; its block is one serial chain (load, QK, softmax, PV), and its N=64 products read
// 6 KB of shared memory for 131,072 multiply-adds. With 128 rows the products run at full rate
// (8 KB for 262,144), but the sums of 128 rows x 512 dims would fill TMEM alone. So a unit takes
// 256 of the output dims and the logits are computed twice, once for each half (3 units of work
// where 2 would do), which leaves room to have two blocks in flight:
//   S[row, key]   = Q[128 x 512] . K_blk^T           (M=128, N=128, K=512)
//   O[row, d]    += P[128 x 128] . V_blk[128 x 256]   (2 x (M=128, N=128, K=128), P from TMEM)
//
// Shared memory (227 KB): six 64-dim chunks of q (96 KB; the last two, dims 384..511, live in TMEM
// as MMA operand, which is also where the rotation is applied on the way) and eight 16 KB slabs
// [128 keys x 64 dims] of K, in two groups of four by block parity. A block first streams the
// four foreign slabs (dims of the other half, used by QK alone) through its group and then its
// own four into the same slots, where PV finds them; meanwhile the other group holds the block
// before for its PV. TMEM: O 256 columns, S 128, P 64, q 64: all 512.
//
// Roles: warps 0-3 store finished units (so the softmax of the next unit need not wait for the
// stores), warp 4 loads K, warp 5 issues the products, warp 6 loads q, warps 8-15 bring q's last
// chunks to TMEM and do the softmax: TMEM lane = row, two warps per 32 rows, 64 keys each.
//
// Bound: the tensor pipe, 71 % active. A block takes about 4,400 cycles, 3,090 of them products
// at full rate; the rest is issue around the waits (the softmax, some 1,000 cycles, runs beside
// them).
// 2,048 tokens of 64 heads at 16,384: 3.74 to 3.81 ms by the clocks, 1,080 to 1,100 TFLOP/s of the
// result's own flops (0.56 to 0.57 of the measured peak, 0.85 to 0.86 with the logits counted
// twice). Short units pay for their change: 64 prompts of 100 tokens 250 us, 4,096 tokens with a
// 128-row window 200 us (303 and 281 while new queries' products began with the dims that go
// through TMEM, those were read 16 bytes a load, and every product had its own code).
#include <cudaTypedefs.h>
#include <math.h>

#include <algorithm>
#include <mutex>

#include "paged_walk.cuh"

namespace dsa {

namespace {

using namespace paged;

constexpr int kRows = 128;      // rows of q in a unit (MMA M)
constexpr int kHalf = kD / 2;   // output dims of a unit
constexpr int kOutWarps = 4;
constexpr int kLoadWarp = 4;
constexpr int kMmaWarp = 5;
constexpr int kQWarp = 6;
constexpr int kSoftWarp0 = 8;
constexpr int kRegsLaunch = 128;
constexpr int kRegsLow = 104;
constexpr int kRegsSoft = 152;   // 256*104 + 256*152 = 512*128, the launch allocation
constexpr int kQSmem = 6;        // chunks of q in shared memory; the last two are in TMEM

// shared memory (the base is 1024-byte aligned: nothing static precedes it)
constexpr uint32_t kSlab = 16384;               // [128 rows x 128 B]
constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffKV = kQSmem * kSlab;
constexpr uint32_t kOffMx = kOffKV + 8 * kSlab;  // [2][128] block maxima of a row's two halves
constexpr uint32_t kOffL1 = kOffMx + 1024;       // [128] sum of the second half
constexpr uint32_t kOffLinv = kOffL1 + 512;      // [128] 1/sum
constexpr uint32_t kOffBar = kOffLinv + 512;
constexpr uint32_t kSmem = kOffBar + 384;
static_assert(kSmem <= 232448, "over the shared memory of one CTA");

// TMEM columns
constexpr uint32_t kOCol = 0;
constexpr uint32_t kSCol = 256;
constexpr uint32_t kPCol = 384;
constexpr uint32_t kQCol = 448;

// D[tmem] (+)= A[tmem] * B[smem]^T; A: lane = row, a column holds two bf16 along K.
__device__ __forceinline__ void mma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// S (+)= Q . K^T over two slabs, dims 64 c .. 64 c + 127, in slots `slot` and the next.
// (Four products a loop, and one copy for the first pair whichever half it is: unrolled whole the
// kernel's code outgrows the instruction caches, which units of few blocks feel. A window of 128
// 238 us, so 209; half the loops, one step for both halves, 218 but 11 % more for a chunk.)
template <bool kTmem>
__device__ __forceinline__ void issue_qk(const uint8_t *smem, uint32_t tmem, int c, int slot,
                                         uint32_t acc0) {
    constexpr uint32_t idesc = idesc_bf16(kRows, kBlock, false, false);
    const uint64_t kd = desc_sw128(smem_u32(smem + kOffKV) + slot * kSlab, 16, 1024);
    const uint64_t qd = desc_sw128(smem_u32(smem + kOffQ) + c * kSlab, 16, 1024);
#pragma unroll 1
    for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            const int k = 4 * e + kk;
            const uint32_t step = e * (kSlab >> 4) + 2 * kk, acc = k > 0 ? 1u : acc0;
            if (kTmem)
                mma_bf16_ta(tmem + kSCol, tmem + kQCol + 8 * k, kd + step, idesc, acc);
            else
                mma_bf16(tmem + kSCol, qd + step, kd + step, idesc, acc);
        }
}

// O (+)= P . V over the block's keys and 128 of the unit's dims (own slabs 2 half, 2 half + 1).
__device__ __forceinline__ void issue_pv(const uint8_t *smem, uint32_t tmem, int par, int half,
                                         uint32_t acc0) {
    constexpr uint32_t idesc = idesc_bf16(kRows, 128, false, true);
    const uint64_t vd =
        desc_sw128(smem_u32(smem + kOffKV) + (4 * par + 2 * half) * kSlab, kSlab, 1024);
#pragma unroll 2
    for (int kk = 0; kk < 8; ++kk)
        mma_bf16_ta(tmem + kOCol + 128 * half, tmem + kPCol + 8 * kk, vd + ((kk * 2048) >> 4),
                    idesc, kk > 0 ? 1u : acc0);
}

// The two softmax warps of a sub-partition (same 32 rows): named barrier 1 + sp, 64 threads.
__device__ __forceinline__ bool vote_any_pair(bool pred, int sp) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n bar.red.or.pred q, %2, 64, p;\n"
        " selp.b32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(pred)), "r"(1 + sp)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ void bar_pair(int sp) {
    asm volatile("bar.sync %0, 64;" ::"r"(1 + sp) : "memory");
}

// 32 bytes to global memory, at a multiple of 32: a whole sector per lane.
__device__ __forceinline__ void store8(void *to, const uint32_t *v) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// 32 bytes from global memory, at a multiple of 32; zeros without `in`.
__device__ __forceinline__ void load8(uint32_t *v, const void *from, bool in) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0;
    if (in)
        asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]),
                       "=r"(v[6]), "=r"(v[7])
                     : "l"(from));
}

// Whether segment i of a run needs other queries than the one before it: the second unit of a
// token group follows the first with the same ones. And whether the segment after x does.
__device__ __forceinline__ bool fresh_q(const Segment &x, int i) { return i == 0 || x.part == 0; }
__device__ __forceinline__ bool last_of_q(const Segment &x, const Walk &w) {
    return x.part == 1 || w.left <= kUnitCost;
}

// Bits [a, b) of a 32-bit word, a and b clamped to 0..32.
__device__ __forceinline__ uint32_t bits_between(int a, int b) {
    a = max(0, min(32, a));
    b = max(0, min(32, b));
    const uint32_t below_b = b == 32 ? 0xFFFFFFFFu : (1u << b) - 1u;
    const uint32_t below_a = a == 32 ? 0xFFFFFFFFu : (1u << a) - 1u;
    return below_b & ~below_a;
}

__device__ __forceinline__ void mask32(uint32_t (&s)[32], uint32_t vis) {
#pragma unroll
    for (int j = 0; j < 32; ++j)
        if (!((vis >> j) & 1u)) s[j] = __float_as_uint(-INFINITY);
}

// 0 when all 32 logits are finite, else NaN.
__device__ __forceinline__ float zero_if_finite32(const uint32_t (&s)[32]) {
    uint64_t t[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 16; ++j)
        t[j & 1] = fma_pair(pair_of(s[2 * j], s[2 * j + 1]), 0, t[j & 1]);
    t[0] = add_pair(t[0], t[1]);
    return first_of(t[0]) + second_of(t[0]);
}

// Bits of the logits that are not finite.
__device__ __forceinline__ uint32_t odd32(const uint32_t (&s)[32]) {
    uint32_t odd = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j)
        if (!(fabsf(__uint_as_float(s[j])) <= 3.4028234e38f)) odd |= 1u << j;
    return odd;
}

__device__ __forceinline__ float max32(const uint32_t (&s)[32]) {
    float t[16];
#pragma unroll
    for (int j = 0; j < 16; ++j)
        t[j] = fmaxf(__uint_as_float(s[j]), __uint_as_float(s[j + 16]));
#pragma unroll
    for (int w = 8; w >= 1; w >>= 1)
#pragma unroll
        for (int j = 0; j < w; ++j) t[j] = fmaxf(t[j], t[j + w]);
    return t[0];
}

// exp2((s - m) c) of 32 products as 16 bf16 pairs; adds the rounded values to l.
__device__ __forceinline__ void exp32(const uint32_t (&s)[32], float c, float m, uint32_t *out,
                                      uint64_t (&l)[2]) {
    const uint64_t c2 = pair_of(c), m2 = pair_of(-m);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const uint64_t x = mul_pair(add_pair(pair_of(s[2 * j], s[2 * j + 1]), m2), c2);
        const __nv_bfloat162 v = __floats2bfloat162_rn(ex2(first_of(x)), ex2(second_of(x)));
        out[j] = *reinterpret_cast<const uint32_t *>(&v);
        l[j & 1] = add_pair(l[j & 1], pair_of(out[j] << 16, out[j] & 0xFFFF0000u));
    }
}

__global__ void __launch_bounds__(kThreads, 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap tm_q,
                       const __grid_constant__ CUtensorMap tm_kv,
                       const __grid_constant__ Params p, const __nv_bfloat16 *__restrict__ q) {
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *sQ = smem + kOffQ;
    uint8_t *sKV = smem + kOffKV;
    float *sMx = reinterpret_cast<float *>(smem + kOffMx);
    float *sL1 = reinterpret_cast<float *>(smem + kOffL1);
    float *sLinv = reinterpret_cast<float *>(smem + kOffLinv);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kOffBar);
    uint64_t *full = bars + 0;      // [2][2] pair of slabs landed, by block parity: the foreign
                                    // ones, then the own ones
    uint64_t *f_free = bars + 4;    // [2][2] pair of foreign slabs used by QK
    uint64_t *v_free = bars + 8;    // [2][2] pair of own slabs used by PV
    uint64_t *pg_full = bars + 12;  // [2] sPages written, by block parity
    uint64_t *q_full = bars + 14;   // q's chunks in shared memory landed
    uint64_t *q_tm = bars + 15;     // q's chunks in TMEM written
    uint64_t *q_free = bars + 16;   // the unit's last QK done
    uint64_t *s_full = bars + 17;
    uint64_t *s_free = bars + 18;
    uint64_t *p_full = bars + 19;
    uint64_t *pv_done = bars + 20;  // PV of a block done: P may be written, O rescaled
    uint64_t *o_full = bars + 21;
    uint64_t *o_free = bars + 22;   // [2] a half of O's columns left by the stores
    uint64_t *stat_full = bars + 24;
    uint64_t *stat_free = bars + 25;  // the stores have read a segment's sums
    uint64_t *drain = bars + 26;    // every product issued is done
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + 27);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    volatile uint32_t *sPages = tmem_holder + 2;             // [2]
    int *sStart = reinterpret_cast<int *>(tmem_holder + 4);  // [5]
    volatile uint32_t *sBlocks = tmem_holder + 1 + kBlocksAt;  // blocks begun

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
        // arrivals a phase takes: a thread per row on o_free and stat_*, 8 softmax warps on
        // s_free, 256 softmax threads on p_full and q_tm, one on the others
        int n = 1;
        uint64_t *bar = bars + lane;
        if (bar == o_free || bar == o_free + 1 || bar == stat_full || bar == stat_free) n = kRows;
        if (bar == s_free) n = 8;
        if (bar == p_full || bar == q_tm) n = 256;
        if (bar <= drain) mbar_init(bar, n);
        if (lane == 31) {
            *abort_flag = 0;
            sStart[4] = 0;
            *sBlocks = 0;
        }
        fence_barrier_init();
    }
    if (warp == kMmaWarp) tmem_alloc(tmem_holder, 512);
    if (tid == 32 * kQWarp) {
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_kv);
    }
    wait_before();
    const int cta = static_cast<int>(blockIdx.x);
    find_run(p, reinterpret_cast<int64_t *>(sKV), sStart);
    const uint32_t tmem = *tmem_holder;

    if (warp < kSoftWarp0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLow));
        if (warp < kOutWarps) {
            // ---------------- finished units to memory. Thread = row.
            const int r = tid;
            const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp * 32) << 16);
            Walk walk(p, sStart);
            Segment x;
            for (int i = 0; walk.next(p, x); ++i) {
                wait_bar(stat_full, i & 1, abort_flag, p.status);
                const float linv = sLinv[r];
                mbar_arrive(stat_free);
                const bool live = wait_bar(o_full, i & 1, abort_flag, p.status);
                tc_fence_after();
                const bool mine = r < x.nrows && live;
                const int slot = 2 * cta + (i > 0);
                const float4 *cs =
                    p.b.cos_sin && half_of(x.part) == 1 && r < x.nrows
                        ? reinterpret_cast<const float4 *>(
                              p.b.cos_sin + int64_t{row_pos(p, x.posf, r)} * kRope)
                        : nullptr;
                __nv_bfloat16 *orow = p.out + (x.row + r) * kD + half_of(x.part) * kHalf;
                // a part's slot: eight dims of a row are 32 bytes, then the next row's, so that a
                // warp writes whole lines
                float *prow = reinterpret_cast<float *>(p.ws + kWsO) + slot * kSlotFloats + r * 8;
#pragma unroll 1
                for (int k = 0; k < kHalf / 32; ++k) {
                    uint32_t o[32];
                    tmem_ld32(lane_base + kOCol + 32 * k, o);
                    tmem_wait_ld();
                    if (k % 4 == 3) {  // the next unit's PV may write this half
                        tc_fence_before();
                        mbar_arrive(&o_free[k / 4]);
                    }
                    if (x.whole) {
                        float v[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(o[j]) * linv;
                        if (cs && k >= 6) {
                            // dims 448..511 turned back by the token's position
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const float4 a = __ldg(cs + 8 * (k - 6) + j);
                                const float v0 = v[4 * j], v1 = v[4 * j + 1];
                                const float v2 = v[4 * j + 2], v3 = v[4 * j + 3];
                                v[4 * j] = v0 * a.x + v1 * a.y;
                                v[4 * j + 1] = v1 * a.x - v0 * a.y;
                                v[4 * j + 2] = v2 * a.z + v3 * a.w;
                                v[4 * j + 3] = v3 * a.z - v2 * a.w;
                            }
                        }
                        uint32_t w[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                            w[j] = *reinterpret_cast<const uint32_t *>(&t);
                        }
                        if (mine) {
                            store8(orow + 32 * k, w);
                            store8(orow + 32 * k + 16, w + 8);
                        }
                    } else if (mine) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            store8(prow + (4 * k + j) * 8 * kRows, o + 8 * j);
                    }
                }
            }
        } else if (warp == kLoadWarp) {
            // ---------------- loader: a block in four steps of two slabs, each one instruction:
            // lane i < np loads page i of the first slab, lane np + i of the second. The block's
            // table entries are read one block ahead.
            const int prows = min(1 << p.b.page_shift, kBlock), np = kBlock / prows;
            const int second = lane >= np, page = second ? lane - np : lane;  // (np: no page)
            uint8_t *const dst0 = sKV + second * kSlab + page * prows * 128;
            const uint64_t pol = policy_evict_normal();  // (each half of the dims reads the keys)
            PageWalk walk(p, sStart);
            int row, row_next = 0, own, own_next = half_of(walk.x.part), g = 0, at = 0;
            bool have = walk.have;
            int32_t e, e_next = walk.next(p, page, prows, np, row_next);
            bool ok = true;
            for (bool more; have; ++g, have = more) {
                e = e_next;
                row = row_next;
                own = own_next;
                own_next = half_of(walk.x.part);
                more = walk.have;
                e_next = walk.next(p, page, prows, np, row_next);
                const int par = g & 1;
                const uint32_t use = (g >> 1) & 1;
                // (every lane, not lane 0 beside its expect_tx: a chunk 3,748 against 3,789 us)
                *sBlocks = static_cast<uint32_t>(g) + 1;
                const uint32_t mask = __ballot_sync(0xFFFFFFFFu, e >= 0);  // both slabs' pages
                const uint32_t bytes = static_cast<uint32_t>(__popc(mask)) * prows * 128;
#pragma unroll 1
                for (at = 0; at < 4; ++at) {
                    // the pair's own slabs of the block two back used by PV; then its foreign
                    // slabs used by QK
                    const int pair = 2 * par + (at & 1);
                    ok = at < 2 ? wait_bar(&v_free[pair], use ^ 1, abort_flag, p.status)
                                : wait_bar(&f_free[pair], use, abort_flag, p.status);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    if (lane == 0) {
                        if (at == 0) {
                            sPages[par] = mask & ((1u << np) - 1u);
                            mbar_arrive(&pg_full[par]);
                        }
                        mbar_expect_tx(&full[pair], bytes);
                    }
                    __syncwarp();
                    const int half = at < 2 ? own ^ 1 : own;  // of the dims
                    if (e >= 0)
                        tma_load_3d(dst0 + 2 * pair * kSlab, &tm_kv, &full[pair],
                                    (4 * half + 2 * (at & 1) + second) * 64, row, e, pol);
                }
                if (!ok) break;
            }
            if (!ok && lane == 0) {
                // gave up in block g before its step `at`: no copy into this CTA's shared memory
                // may still be in flight at exit
                for (int h = 0; h < 2; ++h) {
                    if (at > h || g > 1) drain_wait(&full[2 * (g & 1) + h], at <= h || at > 2 + h);
                    if (g > 0) drain_wait(&full[2 * ((g - 1) & 1) + h], 1);
                }
            }
            __syncwarp();
        } else if (warp == kQWarp) {
            // ---------------- q's chunks in shared memory, as soon as the last ones are read.
            // (Bringing its rows to L2 before that changed nothing.)
            const uint64_t pol_stream = policy_evict_first();
            Walk walk(p, sStart);
            Segment x;
            int loads = 0;
            for (int i = 0; walk.next(p, x); ++i) {
                if (!fresh_q(x, i)) continue;
                if (!wait_bar(q_free, (loads & 1) ^ 1, abort_flag, p.status)) break;
                if (lane == 0) {
                    mbar_expect_tx(q_full, kQSmem * kSlab);
                    for (int c = 0; c < kQSmem; ++c)
                        tma_load_2d(sQ + c * kSlab, &tm_q, q_full, c * 64,
                                    static_cast<int>(x.row), pol_stream);
                }
                ++loads;
            }
            // no copy into this CTA's shared memory may still be in flight at exit
            if (lane == 0 && loads > 0) drain_wait(q_full, (loads - 1) & 1);
            __syncwarp();
        } else if (warp == kMmaWarp) {
            // ---------------- the products, in the order QK foreign (b), PV first half (b - 1),
            // QK own (b), PV second half (b - 1): PV runs where QK would wait, for the own slabs
            // and for the softmax to read S, and the two never alternate MMA by MMA (which
            // costs about 130 cycles a change)
            Walk walk(p, sStart);
            Segment x;
            int g = 0, loads = 0;              // blocks and queries begun
            int ends = 0;                      // segments whose PV is all issued
            bool ok = true, pend = false;      // a block whose PV is to come: is there one, and is
            bool pend_first = false, pend_last = false;  // it its segment's first, last
            // One pass per block, and one more where PV of the last one has no QK to hide behind:
            // before new queries, and at the end.
            bool have = walk.next(p, x), wait_q = have;
            for (int b = 0; ok && (have || pend);) {
                const bool qk = have && !(wait_q && pend);
                const int par = g & 1;
                if (qk) {
                    if (wait_q) {
                        if (!(ok = mbar_wait(q_full, loads & 1, abort_flag, p.status))) break;
                        ++loads;
                        wait_q = false;
                    }
                    // the softmax must have read the block before's S
                    if (!(ok = mbar_wait(s_free, par ^ 1, abort_flag, p.status))) break;
                }
#pragma unroll
                for (int half = 0; half < 2; ++half) {   // of the block: foreign, own
                    if (qk) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (!(ok = mbar_wait(&full[2 * par + h], half, abort_flag, p.status)))
                                break;
                            // (looked at in every block: a flag that says whether this is the
                            // queries' first one costs registers, 271 us where this takes 261)
                            if (h == 1 && (half ^ x.part)) {
                                if (!(ok = mbar_wait(q_tm, (loads - 1) & 1, abort_flag, p.status)))
                                    break;
                            }
                            tc_fence_after();
                            if (elect_one()) {
                                if (h == 0)
                                    issue_qk<false>(smem, tmem, 4 * (half ^ x.part), 4 * par, half);
                                else if (half ^ x.part)
                                    issue_qk<true>(smem, tmem, 6, 4 * par + 2, 1);
                                else
                                    issue_qk<false>(smem, tmem, 2, 4 * par + 2, 1);
                                if (half == 0) mma_commit(&f_free[2 * par + h]);
                            }
                            __syncwarp();
                        }
                        if (!ok) break;
                        if (half == 1 && elect_one()) {
                            mma_commit(s_full);
                            if (b == x.nb - 1 && last_of_q(x, walk)) mma_commit(q_free);
                        }
                        __syncwarp();
                    }
                    if (pend) {
                        if (half == 0) ok = mbar_wait(p_full, (g - 1) & 1, abort_flag, p.status);
                        // the stores of the segment before must have left this half of O
                        if (ok && pend_first && ends > 0)
                            ok = mbar_wait(&o_free[half], (ends - 1) & 1, abort_flag, p.status);
                        if (!ok) break;
                        tc_fence_after();
                        if (elect_one()) {
                            issue_pv(smem, tmem, (g - 1) & 1, half, !pend_first);
                            mma_commit(&v_free[2 * ((g - 1) & 1) + half]);
                            if (half == 1) {
                                mma_commit(pv_done);
                                if (pend_last) mma_commit(o_full);
                            }
                        }
                        __syncwarp();
                    }
                }
                if (!ok) break;
                if (pend && pend_last) ++ends;
                pend = qk;
                if (qk) {
                    ++g;
                    pend_first = b == 0;
                    pend_last = b == x.nb - 1;
                    if (++b == x.nb) {
                        b = 0;
                        have = walk.next(p, x);
                        wait_q = have && x.part == 0;
                    }
                }
            }
            if (elect_one()) {
                mma_commit(drain);
                drain_wait(drain, 0);
            }
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
        // ---------------- softmax, 8 warps: rows of sub-partition sp x keys [64 hh, 64 hh + 64)
        const int sp = warp & 3;
        const int hh = (warp - kSoftWarp0) >> 2;
        const int r = 32 * sp + lane;
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(sp * 32) << 16);
        const int page_shift = min(p.b.page_shift, 7);
        const uint32_t all_pages = (1u << (kBlock >> page_shift)) - 1u;
        Walk walk(p, sStart);
        Segment x;
        int i = 0, g = 0;
        for (; walk.next(p, x); ++i) {
            const bool mine = r < x.nrows;
            const int pos = mine ? row_pos(p, x.posf, r) : x.posl;
            if (fresh_q(x, i)) {
                // q's last two chunks to TMEM, 64 dims by each of a row's two threads, dims
                // 448..511 turned on the way. (The last unit's QK, which read what was there, is
                // done: its last S was read above.)
                const __nv_bfloat16 *src = q + (x.row + r) * kD + 384 + 64 * hh;
                uint32_t v[32];
#pragma unroll
                for (int k = 0; k < 4; ++k) load8(v + 8 * k, src + 16 * k, mine);
                if (hh == 1 && p.b.cos_sin && mine) {
                    const float4 *cs =
                        reinterpret_cast<const float4 *>(p.b.cos_sin + int64_t{pos} * kRope);
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const float4 a = __ldg(cs + k);
                        v[2 * k] = turn_pair(v[2 * k], a.x, a.y);
                        v[2 * k + 1] = turn_pair(v[2 * k + 1], a.z, a.w);
                    }
                }
                tmem_st32(lane_base + kQCol + 32 * hh, v);
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(q_tm);
            }
            uint64_t l[2] = {0, 0};  // two sums each
            float m = kNoMax;
            for (int b = 0; b < x.nb; ++b, ++g) {
                const int par = g & 1;
                const int k0 = (x.blk + b) * kBlock;
                const bool live = __all_sync(
                    0xFFFFFFFFu, mbar_wait(s_full, par, abort_flag, p.status));
                mbar_wait(&pg_full[par], (g >> 1) & 1, abort_flag, p.status);
                tc_fence_after();
                uint32_t s0[32], s1[32];
                tmem_ld32(lane_base + kSCol + 64 * hh, s0);
                tmem_ld32(lane_base + kSCol + 64 * hh + 32, s1);
                const uint32_t pages = sPages[par];
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_free);
                // every row sees every key of the block, unless ...
                if (k0 + kBlock - 1 > x.posf || (p.window > 0 && k0 <= x.posl - p.window) ||
                    pages != all_pages || !live) {
                    const int end = pos - k0 - 64 * hh + 1;   // keys [from, end) of this thread's
                    const int from = p.window > 0 ? end - p.window : 0;
                    uint32_t v0 = bits_between(from, end), v1 = bits_between(from - 32, end - 32);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const bool in = live && ((pages >> ((64 * hh + 16 * k) >> page_shift)) & 1u);
                        const uint32_t half = (k & 1) ? 0xFFFF0000u : 0x0000FFFFu;
                        if (!in && k < 2) v0 &= ~half;
                        if (!in && k >= 2) v1 &= ~half;
                    }
                    // A row of the cache that holds an infinity or NaN makes its logit non-finite
                    // in every row of q. Where a row of q must not see the key, those elements
                    // become zero in the own slabs (0 * inf in PV would reach every row); rows
                    // that do see the key have a NaN probability already, or with a logit of -inf
                    // give it no weight. The sub-partitions' warps, which all see such a key, take
                    // a quarter of the keys each, one at a time: lane = 16-byte piece of its four
                    // slabs.
                    if (__any_sync(0xFFFFFFFFu,
                                   live && !(zero_if_finite32(s0) + zero_if_finite32(s1) == 0.0f))) {
                        const uint32_t mine4 = 0x11111111u << sp;
                        uint32_t odd0 = __reduce_or_sync(0xFFFFFFFFu, odd32(s0)) & mine4;
                        uint32_t odd1 = __reduce_or_sync(0xFFFFFFFFu, odd32(s1)) & mine4;
                        mbar_wait(&full[2 * par], 1, abort_flag, p.status);
                        mbar_wait(&full[2 * par + 1], 1, abort_flag, p.status);
                        uint8_t *tile = sKV + (4 * par + (lane >> 3)) * kSlab + (lane & 7) * 16;
                        while (odd0 | odd1) {
                            int key;
                            if (odd0) {
                                key = __ffs(odd0) - 1;
                                odd0 &= odd0 - 1;
                            } else {
                                key = 32 + __ffs(odd1) - 1;
                                odd1 &= odd1 - 1;
                            }
                            uint4 *at = reinterpret_cast<uint4 *>(tile + (64 * hh + key) * 128);
                            uint4 v = *at;
                            v.x = finite2(v.x);
                            v.y = finite2(v.y);
                            v.z = finite2(v.z);
                            v.w = finite2(v.w);
                            *at = v;
                        }
                        fence_proxy_async_smem();
                    }
                    mask32(s0, v0);
                    mask32(s1, v1);
                }
                const float mx = fmaxf(max32(s0), max32(s1));
                if (vote_any_pair((mx - m) * p.c > kRescale, sp)) {
                    // the row's block maximum from both halves; sums and O rescaled
                    sMx[hh * kRows + r] = mx;
                    bar_pair(sp);
                    const float m_new = fmaxf(m, fmaxf(mx, sMx[(hh ^ 1) * kRows + r]));
                    const float alpha = ex2((m - m_new) * p.c);
                    m = m_new;
                    l[0] = fma_pair(l[0], pair_of(alpha), 0);
                    l[1] = fma_pair(l[1], pair_of(alpha), 0);
                    if (b > 0) {
                        mbar_wait(pv_done, par ^ 1, abort_flag, p.status);
                        tc_fence_after();
#pragma unroll 1
                        for (int k = 0; k < 4; ++k) {
                            uint32_t o[32];
                            const uint32_t col = lane_base + kOCol + 128 * hh + 32 * k;
                            tmem_ld32(col, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
                            tmem_st32(col, o);
                        }
                        tmem_wait_st();
                    }
                }
                // P rounded to bf16; the sums take the rounded values, which PV multiplies
                uint32_t pk[32];
                exp32(s0, p.c, m, pk, l);
                exp32(s1, p.c, m, pk + 16, l);
                mbar_wait(pv_done, par ^ 1, abort_flag, p.status);  // P of the block before is used
                tc_fence_after();
                tmem_st32(lane_base + kPCol + 32 * hh, pk);
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(p_full);
            }
            const uint64_t l2 = add_pair(l[0], l[1]);
            const float sum = first_of(l2) + second_of(l2);
            if (hh == 1) sL1[r] = sum;
            bar_pair(sp);
            if (hh == 0) {
                const float tot = sum + sL1[r];
                // The stores must have taken the segment before's sums: segments of one block
                // can otherwise run two ahead of them, past the phase they wait for.
                if (i > 0) mbar_wait(stat_free, (i - 1) & 1, abort_flag, p.status);
                // a row that saw no key has sum 0 and O 0
                sLinv[r] = tot == 0.0f ? 0.0f : 1.0f / tot;
                if (!x.whole)
                    reinterpret_cast<float2 *>(p.ws + kWsMl)[(2 * cta + (i > 0)) * kMaxRows + r] =
                        make_float2(m, tot);
                mbar_arrive(stat_full);
            }
        }
    }
    __syncthreads();
    if (warp == kMmaWarp) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

std::mutex g_mu;
bool g_done[kMaxDevices];

}  // namespace

int prepare_paged_chunk() {
    const int dev = current_device();
    if (dev < 0) return DSA_ERR_CUDA;
    std::lock_guard<std::mutex> lock(g_mu);
    if (!g_done[dev]) {
        const int rc = prepare_kernel(paged_chunk_kernel, kRegsLaunch, kSmem);
        if (rc != DSA_OK) return rc;
        g_done[dev] = true;
    }
    return DSA_OK;
}

int enqueue_paged_chunk(const CUtensorMap &tm_q, const CUtensorMap &tm_kv,
                        const paged::Params &p, const void *q, int ctas, cudaStream_t s) {
    return launch_overlapped(paged_chunk_kernel, ctas, kThreads, kSmem, s, tm_q, tm_kv, p,
                             static_cast<const __nv_bfloat16 *>(q));
}

}  // namespace dsa
