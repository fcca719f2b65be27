// dsa_paged_attn: attention of a ragged batch's new tokens over their sequences' rows in a
// paged cache.
//
//   out[r,h] = R(-t) sum_u p_u row_u,   p = softmax_u(scale * (R(t) q[r,h]) . row_u)
//
// over the rows u of the token's sequence with t - window < u <= t. One 512-wide row is key
// and value of every head, so the (token, head) rows of q that share keys can be stacked into
// one matrix product whatever token or head they come from.
//
// This file holds the kernel for few rows of q per sequence (single tokens, short bands), the
// join of cut units, and the entry point; paged_chunk.cu the kernel for chunks, paged_walk.cuh
// the list of work that both cut evenly over the SMs. A unit here is up to 64 rows of q:
// floor(64 / heads) whole tokens of a sequence, or 64 of a token's heads and then the rest when
// there are more.
//
// A block (the layout that the window + selected attention of this library uses, with the
// rows loaded by TMA, page by page): everything is transposed so that the 128 keys sit on the
// MMA's M:
//   S^T[key, row]  = K_blk[128 x 512] . Q^T        (M=128, N=64, K=512)
//   O^T[d, row]   += V_blk^T[512 x 128] . P^T       (4 x (M=128, N=64, K=128))
// K_blk and V_blk are one shared-memory tile of eight chunks [128 keys x 64 dims], filled and
// released in pairs (one 128-dim tile of the second product each); a ninth chunk slot lets
// one chunk of the next block land early. Chunk c holds dims 64 ((c + 2) mod 8) ..: the
// rotated dims (448..511) are chunk 5, which the first product reaches in the middle of a
// unit's first block, after other warps have turned that chunk of the queries in place.
//
// Bound: HBM for single tokens (64 heads: 128 flops a byte, against 282 of the machine). One tile
// is all that fits beside q (64 KB) and P, so a block is a chain (PV of the block before frees
// the slots, 1,900 cycles of load latency, the last QK products, 1,000 cycles of softmax). 152
// sequences of 16,384, a unit of 128 blocks for each SM: 441 us from start to join, 5.8 TB/s of
// keys, 85 % of the measured copy rate. One token at 131,072: 44.5 us, 37 without the launch of the
// join; 64 users of up to 8,192: 82.6, 77.4 without. (The compiler spills 100 bytes a thread, 128
// read back, to fit all roles into the launch's 128 registers.)
#include <cudaTypedefs.h>
#include <math.h>

#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "paged_walk.cuh"

namespace dsa {

namespace {

using namespace paged;

// Warpgroups 0-1 (80 registers a thread): the loader warp 0, warps 1-4 that turn the queries,
// the QK-issuing warp 6 and the PV-issuing warp 7 (two issuing warps: a thread that waits
// between MMAs stalls its own issue, not the other's). Warpgroups 2-3 (176): softmax.
// 256*80 + 256*176 = 512*128, the launch allocation (checked before the first launch).
constexpr int kTurnWarp0 = 1;
constexpr int kTurnThreads = 128;
constexpr int kQkWarp = 6;
constexpr int kPvWarp = 7;
constexpr int kSoftWarp0 = 8;
constexpr int kRegsLaunch = 128;
constexpr int kRegsLow = 80;
constexpr int kRegsSoft = 176;
constexpr int kSoftThreads = 256;

constexpr int kRows = 64;     // rows of q in a unit (MMA N)
constexpr int kTurnChunk = 5; // the chunk that holds dims 448..511

__host__ __device__ constexpr int chunk_dim(int c) { return ((c + 2) & 7) * 64; }

// shared memory
constexpr uint32_t kOffQ = 0;                // 8 chunks x [64 rows x 128 B]
constexpr uint32_t kOffKV = 65536;           // 8 chunks x [128 keys x 128 B]
constexpr uint32_t kOffP = 65536 + 131072;   // P^T [128 keys x 64 rows] bf16
constexpr uint32_t kOffX = kOffP + 16384;    // chunk 7 of odd blocks
constexpr uint32_t kOffRed = kOffX + 16384;  // [4][64] block maxima | partial sums
constexpr uint32_t kOffLinv = kOffRed + 1024;// [64] rescale factors | 1/sum
constexpr uint32_t kOffM = kOffLinv + 256;   // [2][64] running maximum, double-buffered
constexpr uint32_t kOffBar = kOffM + 512;
constexpr uint32_t kSmem = kOffBar + 256 + 1024;  // + slack for 1024-B alignment
static_assert(kSmem <= 232448, "over the shared memory of one CTA");
constexpr uint32_t kLbo7Spare = kOffX - (kOffKV + 6 * 16384);  // chunk 6 -> spare chunk 7

// TMEM columns
constexpr uint32_t kSCol = 0;    // S^T, 2 x 64, by block parity
constexpr uint32_t kMCol = 128;  // the running maximum of each row, the same in all lanes
constexpr uint32_t kOCol = 256;  // O^T: 4 d-tiles x 64

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

// ------------------------------------------------------------------ the kernel

__global__ void __launch_bounds__(kThreads, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap tm_q,
                      const __grid_constant__ CUtensorMap tm_kv,
                      const __grid_constant__ Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *sQ = smem + kOffQ;
    uint8_t *sKV = smem + kOffKV;
    uint8_t *sP = smem + kOffP;
    uint8_t *sX = smem + kOffX;
    float *sRed = reinterpret_cast<float *>(smem + kOffRed);
    float *sL = sRed;
    float *sLinv = reinterpret_cast<float *>(smem + kOffLinv);
    float *sAlpha = sLinv;
    float *sM = reinterpret_cast<float *>(smem + kOffM);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kOffBar);
    uint64_t *q_full = bars + 0;
    uint64_t *q_free = bars + 1;
    uint64_t *kv_full = bars + 2;   // [4] chunk pairs 0-2, then chunk 6, landed
    uint64_t *x_full = bars + 6;    // [2] chunk 7 landed, by block parity (usual / spare slot)
    uint64_t *s_free = bars + 8;    // [2] S^T buffer read by the softmax, by block parity
    uint64_t *kv_free = bars + 10;  // [4] chunk pairs 0-2, then chunk 6 (and 7), used by PV
    uint64_t *s_full = bars + 14;
    uint64_t *p_full = bars + 15;
    uint64_t *o_full = bars + 16;
    uint64_t *o_free = bars + 17;
    uint64_t *drain = bars + 18;    // [2] one per issuing warp
    uint64_t *q_turned = bars + 20;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + 21);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    volatile uint32_t *sPages = tmem_holder + 2;  // [2] pages of a block that were loaded
    int *sStart = reinterpret_cast<int *>(tmem_holder + 4);  // [5] start of this CTA's run
    volatile uint32_t *sBlocks = tmem_holder + 1 + kBlocksAt;  // blocks begun

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (warp == 0) {
        // arrivals a phase takes: 128 turning threads on q_turned; 8 softmax warps on s_free
        // and o_free, 256 softmax threads on p_full; on s_full (S^T of a block may be read) QK's
        // commit for it and PV's for the block before; one on the others
        int n = 1;
        uint64_t *bar = bars + lane;
        if (bar == q_turned) n = kTurnThreads;
        if (bar == &s_free[0] || bar == &s_free[1] || bar == o_free) n = 8;
        if (bar == p_full) n = kSoftThreads;
        if (bar == s_full) n = 2;
        if (bar <= q_turned) mbar_init(bar, n);
        if (lane == 31) {
            *abort_flag = 0;
            sStart[4] = 0;
            *sBlocks = 0;
        }
        fence_barrier_init();
    }
    if (warp == kPvWarp) tmem_alloc(tmem_holder, 512);
    if (tid == 32 * kQkWarp) {
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_kv);
    }
    wait_before();
    const int cta = static_cast<int>(blockIdx.x);
    find_run(p, reinterpret_cast<int64_t *>(sKV), sStart);
    const uint32_t tmem = *tmem_holder;

    if (warp < kSoftWarp0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLow));
        if (warp == 0) {
            // ---------------- loader: the pages of each block, chunk by chunk. Lane i < np
            // loads page i; its table entry is read one block ahead. (Rows brought to L2 one to
            // five blocks ahead by bulk prefetches measured 478 to 727 us against 483 for 152
            // sequences of 16K rows: the loads alone keep HBM busy.)
            const int prows = min(1 << p.b.page_shift, kBlock), np = kBlock / prows;
            PageWalk walk(p, sStart);
            int row, row_next = 0, g = 0, m_at = 0;
            bool have = walk.have, alone, alone_next = walk.x.alone;
            int32_t e, e_next = walk.next(p, lane, prows, np, row_next);
            // Keys that no other unit reads pass through L2 without pushing out what is there
            // (q, the parts to be joined): one token at 128K 56 -> 50 us, 32 users of 8K 83 ->
            // 76. Kept for keys that others read: without, a chunk took 18 % longer.
            const uint64_t once = policy_evict_first(), keep = policy_evict_normal();
            bool ok = true;
            for (bool more; have; ++g, have = more) {
                e = e_next;
                row = row_next;
                alone = alone_next;
                alone_next = walk.x.alone;
                more = walk.have;
                e_next = walk.next(p, lane, prows, np, row_next);
                const uint64_t pol = alone ? once : keep;
                const int par = g & 1;
                const uint32_t mask = __ballot_sync(0xFFFFFFFFu, e >= 0);
                const uint32_t bytes = static_cast<uint32_t>(__popc(mask)) * prows * 128;
                const uint32_t off = lane * prows * 128;
                // chunk 7 first, into the slot that the block two back released
                if (lane == 0) {
                    sPages[par] = mask;
                    *sBlocks = static_cast<uint32_t>(g) + 1;
                    mbar_expect_tx(&x_full[par], bytes);
                }
                __syncwarp();
                if (e >= 0)
                    tma_load_3d((par ? sX : sKV + 7 * 16384) + off, &tm_kv, &x_full[par],
                                chunk_dim(7), row, e, pol);
                for (int m = 0; m < 4; ++m) {
                    m_at = m;
                    ok = __all_sync(0xFFFFFFFFu, wait_bar(&kv_free[m], (g & 1) ^ 1, abort_flag,
                                                           p.status));
                    if (!ok) break;
                    if (lane == 0) mbar_expect_tx(&kv_full[m], m < 3 ? 2 * bytes : bytes);
                    __syncwarp();
                    if (e >= 0) {
                        uint8_t *dst = sKV + 2 * m * 16384 + off;
                        tma_load_3d(dst, &tm_kv, &kv_full[m], chunk_dim(2 * m), row, e, pol);
                        if (m < 3)
                            tma_load_3d(dst + 16384, &tm_kv, &kv_full[m], chunk_dim(2 * m + 1),
                                        row, e, pol);
                    }
                }
                if (!ok) break;
            }
            if (!ok && lane == 0) {
                // gave up in block g before its chunk group m_at: no copy into this CTA's
                // shared memory may still be in flight at exit
                for (int m = 0; m < 4; ++m) {
                    const int last = m < m_at ? g : g - 1;
                    if (last >= 0) drain_wait(&kv_full[m], last & 1);
                }
                for (int last = g; last >= 0 && last >= g - 1; --last)
                    drain_wait(&x_full[last & 1], (last >> 1) & 1);
            }
            __syncwarp();
        } else if (warp >= kTurnWarp0 && warp < kTurnWarp0 + kTurnThreads / 32) {
            // ---------------- the queries' rotation, in place: two threads per row, four
            // 16-byte pieces (16 pairs) each; the angles are read before the queries land
            if (p.b.cos_sin) {
                const int t = tid - 32 * kTurnWarp0, r = t >> 1, half = t & 1;
                uint8_t *row = sQ + kTurnChunk * 8192 + r * 128;
                Walk walk(p, sStart);
                Segment x;
                for (int i = 0; walk.next(p, x); ++i) {
                    float4 cs[8];
                    const bool mine = r < x.nrows;
                    if (mine) {
                        const float4 *src =
                            reinterpret_cast<const float4 *>(
                                p.b.cos_sin + int64_t{row_pos(p, x.posf, r)} * kRope) +
                            8 * half;
#pragma unroll
                        for (int k = 0; k < 8; ++k) cs[k] = __ldg(src + k);
                    }
                    if (!wait_bar(q_full, i & 1, abort_flag, p.status)) break;
                    if (mine) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint4 *at =
                                reinterpret_cast<uint4 *>(row + (((4 * half + k) ^ (r & 7)) << 4));
                            uint4 v = *at;
                            v.x = turn_pair(v.x, cs[2 * k].x, cs[2 * k].y);
                            v.y = turn_pair(v.y, cs[2 * k].z, cs[2 * k].w);
                            v.z = turn_pair(v.z, cs[2 * k + 1].x, cs[2 * k + 1].y);
                            v.w = turn_pair(v.w, cs[2 * k + 1].z, cs[2 * k + 1].w);
                            *at = v;
                        }
                    }
                    fence_proxy_async_smem();
                    mbar_arrive(q_turned);
                }
            }
        } else if (warp == kQkWarp) {
            // ---------------- QK issuer: S^T = K_blk . Q^T, chunk pair by chunk pair as the
            // rows land. It loads the unit's queries itself as soon as its own MMAs have read
            // the previous ones.
            constexpr uint32_t idesc_qk = idesc_bf16(kBlock, kRows, false, false);
            const uint64_t ad0 = desc_sw128(smem_u32(sKV), 16, 1024);
            const uint64_t adx = desc_sw128(smem_u32(sX), 16, 1024);
            const uint64_t bd0 = desc_sw128(smem_u32(sQ), 16, 1024);
            const uint64_t pol_stream = policy_evict_first();
            Walk walk(p, sStart);
            Segment x;
            int i = 0, g = 0, last_q = -1;
            bool ok = true;
            for (; ok && walk.next(p, x); ++i) {
                if (!(ok = wait_bar(q_free, (i & 1) ^ 1, abort_flag, p.status))) break;
                if (elect_one()) {
                    mbar_expect_tx(q_full, 65536);
                    for (int c = 0; c < 8; ++c)
                        tma_load_2d(sQ + c * 8192, &tm_q, q_full, chunk_dim(c),
                                    static_cast<int>(x.row), pol_stream);
                }
                last_q = i;
                if (!(ok = wait_bar(q_full, i & 1, abort_flag, p.status))) break;
                tc_fence_after();
                for (int b = 0; b < x.nb && ok; ++b, ++g) {
                    // S^T is double-buffered: QK of a block may run while the softmax of the
                    // block before it does
                    const int par = g & 1;
                    if (!(ok = wait_bar(&s_free[par], ((g >> 1) & 1) ^ 1, abort_flag, p.status)))
                        break;
                    const uint32_t s_col = tmem + kSCol + 64 * par;
                    if (!(ok = wait_bar(&x_full[par], (g >> 1) & 1, abort_flag, p.status))) break;
                    tc_fence_after();
                    if (elect_one()) {
                        const uint64_t ad = par ? adx : ad0 + ((7 * 16384) >> 4);
                        const uint64_t bd = bd0 + ((7 * 8192) >> 4);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_bf16(s_col, ad + 2 * kk, bd + 2 * kk, idesc_qk, kk != 0);
                    }
                    __syncwarp();
#pragma unroll 1
                    for (int m = 0; m < 4; ++m) {
                        if (!(ok = wait_bar(&kv_full[m], g & 1, abort_flag, p.status))) break;
                        if (m == 2 && b == 0 && p.b.cos_sin &&
                            !(ok = wait_bar(q_turned, i & 1, abort_flag, p.status)))
                            break;
                        tc_fence_after();
                        if (elect_one()) {
                            const uint64_t ad = ad0 + ((2 * m * 16384) >> 4);
                            const uint64_t bd = bd0 + ((2 * m * 8192) >> 4);
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                mma_bf16(s_col, ad + 2 * kk, bd + 2 * kk, idesc_qk, 1u);
                            if (m < 3) {
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk)
                                    mma_bf16(s_col, ad + (16384 >> 4) + 2 * kk,
                                             bd + (8192 >> 4) + 2 * kk, idesc_qk, 1u);
                            } else {
                                mma_commit(s_full);
                                if (b == x.nb - 1) mma_commit(q_free);
                            }
                        }
                        __syncwarp();
                    }
                }
            }
            if (elect_one()) {
                mma_commit(&drain[0]);
                drain_wait(&drain[0], 0);
                // no copy into this CTA's shared memory may still be in flight at exit
                if (last_q >= 0) drain_wait(q_full, last_q & 1);
            }
            __syncwarp();
        } else if (warp == kPvWarp) {
            // ---------------- PV issuer: O^T += V_blk^T . P^T, one d-tile at a time
            constexpr uint32_t idesc_pv = idesc_bf16(128, kRows, true, true);
            Walk walk(p, sStart);
            Segment x;
            int i = 0, g = 0;
            bool ok = true;
            if (lane == 0) mbar_arrive(s_full);  // no PV precedes the first block
            __syncwarp();
            for (; ok && walk.next(p, x); ++i) {
                for (int b = 0; b < x.nb && ok; ++b, ++g) {
                    if (!(ok = wait_bar(p_full, g & 1, abort_flag, p.status))) break;
                    tc_fence_after();
                    if (b == 0 && i > 0) {
                        // the epilogue of the previous unit must have read O^T
                        if (!(ok = wait_bar(o_free, (i - 1) & 1, abort_flag, p.status))) break;
                        tc_fence_after();
                    }
                    const uint32_t acc0 = b > 0;
                    const uint32_t lbo3 = (g & 1) ? kLbo7Spare : 16384u;
                    if (elect_one()) {
                        // (one tile's code four times over: 152 sequences of 16,384 457 -> 445 us
                        // against four copies)
#pragma unroll 1
                        for (int m = 0; m < 4; ++m) {
#pragma unroll
                            for (int kk = 0; kk < 8; ++kk)
                                mma_bf16(tmem + kOCol + 64 * m,
                                         desc_sw128(smem_u32(sKV + 2 * m * 16384 + kk * 2048),
                                                    m < 3 ? 16384u : lbo3, 1024),
                                         desc_sw128(smem_u32(sP + kk * 2048), 8192, 1024),
                                         idesc_pv, kk > 0 ? 1u : acc0);
                            mma_commit(&kv_free[m]);
                        }
                        mma_commit(s_full);
                        if (b == x.nb - 1) mma_commit(o_full);
                    }
                    __syncwarp();
                }
            }
            if (elect_one()) {
                mma_commit(&drain[1]);
                drain_wait(&drain[1], 0);
            }
            __syncwarp();
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
        const int page_shift = min(p.b.page_shift, 7);
        const uint32_t all_pages = (1u << (kBlock >> page_shift)) - 1u;
        Walk walk(p, sStart);
        Segment x;
        int i = 0, g = 0, cur = 0;
        for (; walk.next(p, x); ++i) {
            float l[32];
#pragma unroll
            for (int h = 0; h < 32; ++h) l[h] = 0.0f;
            if (sp == 0) sM[cur * 64 + hb + lane] = kNoMax;
            {
                uint32_t none[32];
#pragma unroll
                for (int h = 0; h < 32; ++h) none[h] = __float_as_uint(kNoMax);
                tmem_st32(lane_base + kMCol + hb, none);
                tmem_wait_st();
            }
            bar_group(hh);
            for (int b = 0; b < x.nb; ++b, ++g) {
                const int par = g & 1;
                const int k0 = (x.blk + b) * kBlock;
                // S^T of this block is ready and the previous block's PV is done with P and O^T
                const bool live = __all_sync(
                    0xFFFFFFFFu, mbar_wait(s_full, g & 1, abort_flag, p.status));
                // (complete since QK of this block waited for it: orders sPages before here)
                mbar_wait(&x_full[par], (g >> 1) & 1, abort_flag, p.status);
                tc_fence_after();
                uint32_t sa[32], mv[32];
                tmem_ld32(lane_base + kMCol + hb, mv);
                if (live) tmem_ld32(lane_base + kSCol + 64 * par + hb, sa);
                const uint32_t pages = sPages[par];
                tmem_wait_ld();
                // this S^T buffer may take the QK of the block after next
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_free[par]);
                // every row sees every key of the block, unless ...
                if (k0 + kBlock - 1 > x.posf || (p.window > 0 && k0 <= x.posl - p.window) ||
                    pages != all_pages || !live) {
                    // rows [ra, rb) of the unit see key k0 + kl: their token is not before it
                    // and less than `window` after it
                    const int64_t ahead = int64_t{k0} + kl - x.posf;
                    const int ta = static_cast<int>(max(int64_t{0}, min(ahead, int64_t{64})));
                    const int64_t gone = p.window > 0 ? ahead + p.window : 64;
                    const int tb = static_cast<int>(max(int64_t{0}, min(gone, int64_t{64})));
                    const int ra = min(64, ta * p.rpt);
                    int rb = min(64, tb * p.rpt);
                    if (!((pages >> (kl >> page_shift)) & 1u) || !live) rb = 0;
                    // A row of the cache that holds an infinity or NaN makes its logit non-finite
                    // in every row of q. Where a row of q must not see the key, those elements
                    // become zero in the tile (0 * inf in PV would reach every row); rows that
                    // do see the key have a NaN probability already, or with a logit of -inf
                    // give it no weight. A key at a time: lane = 16-byte piece of four of its
                    // chunks.
                    const int a = max(0, min(32, ra - hb)), e = max(0, min(32, rb - hb));
                    const uint32_t below_e = e == 32 ? 0xFFFFFFFFu : (1u << e) - 1u;
                    const uint32_t below_a = a == 32 ? 0xFFFFFFFFu : (1u << a) - 1u;
                    const uint32_t vis = below_e & ~below_a;
                    float t4[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // NaN if any is not finite
#pragma unroll
                    for (int h = 0; h < 32; ++h)
                        t4[h & 3] = fmaf(__uint_as_float(sa[h]), 0.0f, t4[h & 3]);
                    const bool odd = !((t4[0] + t4[1]) + (t4[2] + t4[3]) == 0.0f);
#pragma unroll
                    for (int h = 0; h < 32; ++h)
                        if (!((vis >> h) & 1u)) sa[h] = __float_as_uint(-INFINITY);
                    uint32_t keys =
                        __ballot_sync(0xFFFFFFFFu, odd && live && (ra > 0 || rb < x.nrows));
                    if (keys) {
                        for (int m = 0; m < 4; ++m)
                            mbar_wait(&kv_full[m], g & 1, abort_flag, p.status);
                        const int c = 4 * hh + (lane >> 3);
                        uint8_t *tile =
                            (c == 7 && par ? sX : sKV + c * 16384) + sp * 4096 + (lane & 7) * 16;
                        for (; keys; keys &= keys - 1) {
                            uint4 *at = reinterpret_cast<uint4 *>(tile + (__ffs(keys) - 1) * 128);
                            uint4 v = *at;
                            v.x = finite2(v.x);
                            v.y = finite2(v.y);
                            v.z = finite2(v.z);
                            v.w = finite2(v.w);
                            *at = v;
                        }
                    }
                }
                // xv = (product - running maximum) * c: decides the rescale, feeds exp2
                float xv[32];
                float xmax;
                {
#pragma unroll
                    for (int h = 0; h < 32; ++h)
                        xv[h] = (__uint_as_float(sa[h]) - __uint_as_float(mv[h])) * p.c;
                    float t16[16];
#pragma unroll
                    for (int h = 0; h < 16; ++h) t16[h] = fmaxf(xv[h], xv[h + 16]);
#pragma unroll
                    for (int w = 8; w >= 1; w >>= 1)
#pragma unroll
                        for (int h = 0; h < w; ++h) t16[h] = fmaxf(t16[h], t16[h + w]);
                    xmax = t16[0];
                }
                if (vote_any_group(xmax > kRescale, hh)) {
                    // exact block maxima -> new running maximum; sums and O^T rescaled
#pragma unroll
                    for (int h = 0; h < 32; ++h) {
                        const float wm = redux_max(__uint_as_float(sa[h]));
                        if (lane == h) sRed[sp * 64 + hb + h] = wm;
                    }
                    bar_group(hh);
                    if (sp == 0) {
                        const int r = hb + lane;
                        const float bm = fmaxf(fmaxf(sRed[r], sRed[64 + r]),
                                               fmaxf(sRed[128 + r], sRed[192 + r]));
                        const float m_old = sM[cur * 64 + r];
                        const float m_new = fmaxf(m_old, bm);
                        sM[(cur ^ 1) * 64 + r] = m_new;
                        sAlpha[r] = ex2((m_old - m_new) * p.c);
                    }
                    bar_group(hh);
                    cur ^= 1;
                    const float *m_now = sM + cur * 64 + hb;
#pragma unroll
                    for (int h = 0; h < 32; ++h) {
                        mv[h] = __float_as_uint(m_now[h]);
                        l[h] *= sAlpha[hb + h];
                        xv[h] = (__uint_as_float(sa[h]) - m_now[h]) * p.c;
                    }
                    tmem_st32(lane_base + kMCol + hb, mv);
                    tmem_wait_st();
                    if (b > 0 && live) {
#pragma unroll 1
                        for (int m = 0; m < 4; ++m) {
                            uint32_t oa[32];
                            const uint32_t col = lane_base + kOCol + 64 * m + hb;
                            tmem_ld32(col, oa);
                            tmem_wait_ld();
#pragma unroll
                            for (int h = 0; h < 32; ++h)
                                oa[h] = __float_as_uint(__uint_as_float(oa[h]) * sAlpha[hb + h]);
                            tmem_st32(col, oa);
                        }
                        tmem_wait_st();
                    }
                }
                // this thread's 32 rows of P^T for key kl: four swizzled 16-byte pieces. The
                // sums take P as rounded to bf16, the values that PV multiplies.
                {
                    uint8_t *prow = sP + kl * 128;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t pk[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const __nv_bfloat162 v = __floats2bfloat162_rn(
                                ex2(xv[8 * q + 2 * e]), ex2(xv[8 * q + 2 * e + 1]));
                            pk[e] = *reinterpret_cast<const uint32_t *>(&v);
                            l[8 * q + 2 * e] += bf16lo(pk[e]);
                            l[8 * q + 2 * e + 1] += bf16hi(pk[e]);
                        }
                        *reinterpret_cast<uint4 *>(prow + (((4 * hh + q) ^ (kl & 7)) << 4)) =
                            make_uint4(pk[0], pk[1], pk[2], pk[3]);
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                mbar_arrive(p_full);
            }
            // ---- end of the segment: sums over the keys. Transpose-reduce the 32 partial
            // sums across the warp: lane ends with the warp's total for row hb + lane
#pragma unroll
            for (int w = 16; w >= 1; w >>= 1) {
                const bool up = (lane & w) != 0;
#pragma unroll
                for (int h = 0; h < w; ++h) {
                    const float send = up ? l[h] : l[h + w];
                    const float keep = up ? l[h + w] : l[h];
                    l[h] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, w);
                }
            }
            sL[sp * 64 + hb + lane] = l[0];
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
                        make_float2(sM[cur * 64 + r], tot);
            }
            bar_group(hh);
            // O^T into registers one d-tile at a time: lane holds dim 128 m' + 32 sp + lane of
            // rows hb .. hb + 31, so a warp writes 32 consecutive dims of each row
            const bool live = mbar_wait(o_full, i & 1, abort_flag, p.status);
            tc_fence_after();
            const int rows = min(32, x.nrows - hb);
            if (x.whole) {
                __nv_bfloat16 *orow = p.out + (x.row + hb) * kD + 32 * sp + lane;
                float linv[32];
#pragma unroll
                for (int h = 0; h < 32; h += 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(&sLinv[hb + h]);
                    linv[h] = v.x;
                    linv[h + 1] = v.y;
                    linv[h + 2] = v.z;
                    linv[h + 3] = v.w;
                }
#pragma unroll 1
                for (int m = 0; m < 4; ++m) {
                    uint32_t oa[32];
                    if (!live) break;
                    tmem_ld32(lane_base + kOCol + 64 * m + hb, oa);
                    tmem_wait_ld();
                    __nv_bfloat16 *o = orow + chunk_dim(2 * m);
                    if (p.b.cos_sin && m == kTurnChunk / 2 && sp >= 2) {
                        // turned back by the token's position; a pair is in two adjacent lanes
                        const float2 *cs = reinterpret_cast<const float2 *>(p.b.cos_sin) +
                                           ((sp - 2) * 16 + (lane >> 1));
                        // (a unit of one token's heads has one position)
                        int pos = p.tpu == 1 ? x.posf : x.posf + hb / p.rpt;
                        int left = p.tpu == 1 ? 32 : p.rpt - hb % p.rpt;  // rows at pos
                        float2 a = __ldg(cs + int64_t{pos <= x.posl ? pos : x.posl} * kRopePairs);
#pragma unroll
                        for (int h = 0; h < 32; ++h) {
                            const float v = __uint_as_float(oa[h]) * linv[h];
                            const float w = __shfl_xor_sync(0xFFFFFFFFu, v, 1);
                            if (h < rows) {
                                if (left == 0) {
                                    ++pos;
                                    left = p.rpt;
                                    a = __ldg(cs + int64_t{pos} * kRopePairs);
                                }
                                --left;
                                o[h * kD] = __float2bfloat16_rn(v * a.x + (lane & 1 ? -w : w) * a.y);
                            }
                        }
                    } else {
#pragma unroll
                        for (int h = 0; h < 32; ++h)
                            if (h < rows)
                                o[h * kD] =
                                    __float2bfloat16_rn(__uint_as_float(oa[h]) * linv[h]);
                    }
                }
            } else {
                float *orow = reinterpret_cast<float *>(p.ws + kWsO) +
                              (int64_t{slot} * kRows + hb) * kD + 32 * sp + lane;
#pragma unroll 1
                for (int m = 0; m < 4; ++m) {
                    uint32_t oa[32];
                    if (!live) break;
                    tmem_ld32(lane_base + kOCol + 64 * m + hb, oa);
                    tmem_wait_ld();
                    float *o = orow + chunk_dim(2 * m);
#pragma unroll
                    for (int h = 0; h < 32; ++h)
                        if (h < rows) o[h * kD] = __uint_as_float(oa[h]);
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

// ------------------------------------------------------------------ the join

// out[row] = sum_p O_p w_p / sum_p l_p w_p, w_p = 2^((m_p - M) c), M = max_p m_p, over the parts of a
// unit, always added in the same order. A warp takes one row (or 32 rows x 32 dims of the chunk
// kernel's units): up to kFew parts, what a run's ends leave of most batches, with all their
// loads in flight at once. A row of more parts is taken in pieces of 32 dims, one per warp: four
// groups of eight lanes share the parts, eight loads in flight each, so that one unit of 147
// parts (a single token at 128K) takes a few microseconds too.
constexpr int kJoinWarps = 8;
constexpr int kFew = 32;       // of 512 dims
constexpr int kFewHalf = 16;   // of 256 dims

__device__ __forceinline__ void store_joined(const Params &p, const JoinDesc &d, int r, int dim,
                                             float4 acc, float inv) {
    acc.x *= inv;
    acc.y *= inv;
    acc.z *= inv;
    acc.w *= inv;
    if (p.b.cos_sin && dim >= kD - kRope) {
        const float4 a = __ldg(reinterpret_cast<const float4 *>(
            p.b.cos_sin + int64_t{row_pos(p, d.pos, r)} * kRope + (dim - (kD - kRope))));
        acc = make_float4(acc.x * a.x + acc.y * a.y, acc.y * a.x - acc.x * a.y,
                          acc.z * a.z + acc.w * a.w, acc.w * a.z - acc.z * a.w);
    }
    const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x, acc.y);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z, acc.w);
    *reinterpret_cast<uint2 *>(p.out + (d.row + r) * kD + dim) = make_uint2(
        *reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
}

__device__ __forceinline__ void add_scaled(float4 &acc, float4 o, float w) {
    acc.x = fmaf(o.x, w, acc.x);
    acc.y = fmaf(o.y, w, acc.y);
    acc.z = fmaf(o.z, w, acc.z);
    acc.w = fmaf(o.w, w, acc.w);
}

template <int kDims>
__global__ void __launch_bounds__(kJoinWarps * 32)
    paged_join_kernel(const __grid_constant__ Params p, int ctas) {
    constexpr int kWords = (kMaxCtas + 31) / 32, kLoads = kDims / 128;
    constexpr int kFewest = kDims == kD ? kFew : kFewHalf;
    __shared__ JoinDesc descs[kMaxCtas];
    __shared__ int owner[kMaxCtas];           // the CTA a descriptor is of
    __shared__ int count[2][kWords];
    __shared__ float weight[kJoinWarps][kWords * 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    wait_before();
    // the units of few parts first, then the others
    JoinDesc d = {};
    if (tid < ctas) d = reinterpret_cast<const JoinDesc *>(p.ws + kWsDesc)[tid];
    const uint32_t few = __ballot_sync(0xFFFFFFFFu, d.parts > 0 && d.parts <= kFewest);
    const uint32_t many = __ballot_sync(0xFFFFFFFFu, d.parts > kFewest);
    if (lane == 0 && warp < kWords) {
        count[0][warp] = __popc(few);
        count[1][warp] = __popc(many);
    }
    __syncthreads();
    int before[2] = {0, 0}, n[2] = {0, 0};
    for (int k = 0; k < 2; ++k)
        for (int w = 0; w < kWords; ++w) {
            if (w < warp) before[k] += count[k][w];
            n[k] += count[k][w];
        }
    if (d.parts > 0) {
        const int k = d.parts > kFewest;
        const uint32_t below = (k ? many : few) & ((1u << lane) - 1u);
        const int at = (k ? n[0] : 0) + before[k] + __popc(below);
        descs[at] = d;
        owner[at] = tid;
    }
    __syncthreads();
    const float *const parts_o = reinterpret_cast<const float *>(p.ws + kWsO);
    const float2 *const parts_ml = reinterpret_cast<const float2 *>(p.ws + kWsMl);
    const int stride = static_cast<int>(gridDim.x) * kJoinWarps;
    const int first = static_cast<int>(blockIdx.x) * kJoinWarps + warp;

    if constexpr (kDims == kD) {
        for (int it = first; it < n[0] * p.rows; it += stride) {
            const JoinDesc &u = descs[it / p.rows];
            const int cta = owner[it / p.rows], r = it % p.rows;
            if (r >= u.nrows) continue;
            auto slot_of = [&](int k) { return k == 0 ? 2 * cta + u.slot0 : 2 * (cta + k); };
            // lane k holds part k's maximum and sum
            const float2 ml = lane < u.parts ? parts_ml[slot_of(lane) * kMaxRows + r]
                                             : make_float2(kNoMax, 0.0f);
            const float wt = ex2((ml.x - redux_max(ml.x)) * p.c);
            float sum = lane < u.parts ? ml.y * wt : 0.0f;
#pragma unroll
            for (int w = 16; w >= 1; w >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, w);
            float4 acc[kLoads] = {};
#pragma unroll 4
            for (int k = 0; k < u.parts; ++k) {
                const float w = __shfl_sync(0xFFFFFFFFu, wt, k);
                const float *o = parts_o + slot_of(k) * kSlotFloats + r * kDims + 4 * lane;
#pragma unroll
                for (int j = 0; j < kLoads; ++j)
                    add_scaled(acc[j], *reinterpret_cast<const float4 *>(o + 128 * j), w);
            }
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
            for (int j = 0; j < kLoads; ++j)
                store_joined(p, u, r, 128 * j + 4 * lane, acc[j], inv);
        }
    } else {
        // 32 rows x 32 dims, lane = row: the slots' layout gives whole lines
        const int pieces = (kChunkRows / 32) * (kDims / 32);  // of a unit
        for (int it = first; it < n[0] * pieces; it += stride) {
            const JoinDesc &u = descs[it / pieces];
            const int cta = owner[it / pieces];
            const int r = it % pieces / (kDims / 32) * 32 + lane, dim0 = it % (kDims / 32) * 32;
            if (r - lane >= u.nrows) continue;
            auto slot_of = [&](int k) { return k == 0 ? 2 * cta + u.slot0 : 2 * (cta + k); };
            float M = kNoMax, sum = 0.0f;
#pragma unroll 4
            for (int k = 0; k < u.parts; ++k)
                M = fmaxf(M, parts_ml[slot_of(k) * kMaxRows + r].x);
            float4 acc[8] = {};
#pragma unroll 2
            for (int k = 0; k < u.parts; ++k) {
                const int slot = slot_of(k);
                const float2 ml = parts_ml[slot * kMaxRows + r];
                const float w = ex2((ml.x - M) * p.c);
                sum += ml.y * w;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    add_scaled(acc[j],
                               *reinterpret_cast<const float4 *>(
                                   parts_o + slot * kSlotFloats +
                                   slot_at(kChunkRows, r, dim0 + 4 * j)),
                               w);
            }
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            if (r < u.nrows) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    store_joined(p, u, r, half_of(u.part) * kDims + dim0 + 4 * j, acc[j], inv);
            }
        }
    }

    const int pieces = p.rows * (kDims / 32);  // of a unit
    for (int it = first; it < n[1] * pieces; it += stride) {
        const JoinDesc &u = descs[n[0] + it / pieces];
        const int cta = owner[n[0] + it / pieces];
        const int r = it % pieces / (kDims / 32), dim0 = it % (kDims / 32) * 32;
        if (r >= u.nrows) continue;
        auto slot_of = [&](int k) { return k == 0 ? 2 * cta + u.slot0 : 2 * (cta + k); };
        float2 v[kWords];
        float M = kNoMax;
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
            const int k = 32 * j + lane;
            v[j] = k < u.parts ? parts_ml[slot_of(k) * kMaxRows + r] : make_float2(kNoMax, 0.0f);
            M = fmaxf(M, v[j].x);
        }
        M = redux_max(M);
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
            const float w = ex2((v[j].x - M) * p.c);
            weight[warp][32 * j + lane] = w;
            sum += v[j].y * w;
        }
#pragma unroll
        for (int w = 16; w >= 1; w >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, w);
        __syncwarp();
        const int grp = lane >> 3, dim = dim0 + 4 * (lane & 7);
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
        for (int k = grp; k < u.parts; k += 4)
            add_scaled(acc,
                       *reinterpret_cast<const float4 *>(
                           parts_o + slot_of(k) * kSlotFloats +
                           (kDims == kD ? r * kDims + dim : slot_at(kChunkRows, r, dim))),
                       weight[warp][k]);
        __syncwarp();  // the weights are read
#pragma unroll
        for (int w = 8; w <= 16; w <<= 1) {
            acc.x += __shfl_xor_sync(0xFFFFFFFFu, acc.x, w);
            acc.y += __shfl_xor_sync(0xFFFFFFFFu, acc.y, w);
            acc.z += __shfl_xor_sync(0xFFFFFFFFu, acc.z, w);
            acc.w += __shfl_xor_sync(0xFFFFFFFFu, acc.w, w);
        }
        if (grp == 0)
            store_joined(p, u, r, (kDims < kD ? half_of(u.part) * kDims : 0) + dim, acc,
                         sum == 0.0f ? 0.0f : 1.0f / sum);
    }
}

// ------------------------------------------------------------------ host

std::mutex g_mu;
int g_sms[kMaxDevices];   // 0: not set up yet

// Places that a CTA's run may have (of a GB300's 152), from the sizes alone (lengths are the
// device's): the kernels count them in 32 bits.
int64_t run_bound(const Params &p) {
    const int64_t groups = std::min(p.b.n_new, p.b.n_new / p.tpu + p.b.n_seqs);
    const int64_t keys = p.window > 0 ? std::min(p.b.len_limit, p.window + p.tpu) : p.b.len_limit;
    return groups * p.upt * (keys / kBlock + 2 + kUnitCost) / kMaxCtas + 1;
}

// Per-device one-time set-up. A failure is not kept: it may pass (memory for the module's code).
int setup(int *sms) {
    const int dev = current_device();
    if (dev < 0) return DSA_ERR_CUDA;
    std::lock_guard<std::mutex> lock(g_mu);
    if (!g_sms[dev]) {
        const int n = sm_count();
        const int rc = n > 0 ? prepare_kernel(paged_attn_kernel, kRegsLaunch, kSmem) : DSA_ERR_CUDA;
        if (rc != DSA_OK) return rc;
        g_sms[dev] = n;
    }
    *sms = g_sms[dev];
    return DSA_OK;
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
    Params p;
    int rc = check_paged_batch(n_new, new_start, seq_len, n_seqs, page_table, max_pages, pages,
                               n_pages, page_stride, page_size, cos_sin, n_pos, &p.b);
    if (rc != DSA_OK) return rc;
    const float c = scale * 1.4426950408889634f;
    if (heads < 1 || heads > DSA_MAX_PAGED_HEADS || window < 0 || !(scale > 0.0f) || isinf(c) ||
        n_new * heads > (int64_t{1} << 31) - 1)
        return DSA_ERR_SHAPE;
    const uintptr_t qa = reinterpret_cast<uintptr_t>(q), oa = reinterpret_cast<uintptr_t>(out);
    const uintptr_t bytes = static_cast<uintptr_t>(n_new) * heads * kD * 2;
    auto overlap = [](uintptr_t a, uintptr_t na, uintptr_t b, uintptr_t nb) {
        return a < b + nb && b < a + na;
    };
    if (overlap(qa, bytes, oa, bytes) || touches_pages(p.b, pages, out, bytes)) return DSA_ERR_ARG;
    p.heads = heads;
    // The chunk kernel from an average of more than 256 rows of q per sequence on. Below, a unit
    // of 64 rows reads the keys at most four times and does not compute the logits twice. Single
    // and chunk kernel (us): 32 sequences of 8,192 with 64 rows 67 / 120, 128 rows 122 / 125,
    // 256 rows 222 / 233, 512 rows 398 / 401; 4 of 1,024 with 64 rows 16 / 22, 256 rows 20 / 24;
    // 16 of up to 16,384 with 160 on average 84 / 97; 64 prompts of 100 tokens (6,400 rows) 460 /
    // 249; one of 2,048 tokens at 16,384 4,360 / 3,796; 32 of one token of 128 heads 54 / 58.
    // (An average: 64 single tokens of up to 8,192 beside a prompt of 512 all go to the chunk
    // kernel, 187 us where the two apart take 83 and 52.)
    // It loads q and stores out 32 bytes at a time, so arrays that begin between (views at an odd
    // multiple of eight elements) are left to the other kernel, which is right for every batch.
    const bool chunk = n_new * heads > int64_t{n_seqs} * 256 && ((qa | oa) & 31u) == 0;
    if (chunk) {
        p.rows = kChunkRows;
        p.tpu = kChunkRows / heads;
        p.upt = 2;
        p.row_step = 0;
    } else {
        p.rows = kRows;
        p.tpu = heads <= kRows ? kRows / heads : 1;
        p.upt = (heads + kRows - 1) / kRows;
        p.row_step = kRows;
    }
    p.rpt = std::min(heads, p.rows);
    // a window no shorter than any sequence is no window
    p.window = window >= p.b.len_limit ? 0 : window;
    if (run_bound(p) > (int64_t{1} << 31) - 1) return DSA_ERR_SHAPE;
    if (!workspace || !aligned16(workspace) || workspace_bytes < DSA_PAGED_WORKSPACE_BYTES)
        return DSA_ERR_SCRATCH;
    const uintptr_t wa = reinterpret_cast<uintptr_t>(workspace), used = DSA_PAGED_WORKSPACE_BYTES;
    if (overlap(wa, used, qa, bytes) || overlap(wa, used, oa, bytes) ||
        touches_pages(p.b, pages, workspace, used))
        return DSA_ERR_ARG;
    p.out = static_cast<__nv_bfloat16 *>(out);
    // whole lines (the caller's buffer begins on 16 bytes at least)
    p.ws = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(workspace) + (kWsAlign - 1)) &
                                       ~uintptr_t{kWsAlign - 1});
    p.c = c;
    p.status = dev_status;
    int sms = 0;
    rc = setup(&sms);
    if (rc == DSA_OK && chunk) rc = prepare_paged_chunk();
    if (rc != DSA_OK) return rc;
    CUtensorMap tm_q, tm_kv;
    if (!make_tmap_bf16(&tm_q, q, kD, static_cast<uint64_t>(n_new) * heads, kD * 2, 64,
                        p.rows) ||
        !make_tmap_pages(&tm_kv, pages, p.b))
        return DSA_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int ctas = std::min(sms, kMaxCtas);
    rc = chunk ? enqueue_paged_chunk(tm_q, tm_kv, p, q, ctas, s)
               : launch_overlapped(paged_attn_kernel, ctas, kThreads, kSmem, s, tm_q, tm_kv, p);
    if (rc != DSA_OK) return rc;
    return chunk ? launch_overlapped(paged_join_kernel<kD / 2>, 4 * ctas, kJoinWarps * 32, 0, s,
                                     p, ctas)
                 : launch_overlapped(paged_join_kernel<kD>, 4 * ctas, kJoinWarps * 32, 0, s, p,
                                     ctas);
}
