// What the two kernels of dsa_paged_attn and that of dsa_paged_q4_attn share: the list of units and
// key blocks that is cut evenly over the CTAs, the workspace in which the parts of a cut unit meet,
// and small helpers.
//
// Work. A unit is a few whole tokens of one sequence (or part of one token's heads): rows of q
// that attend over the same rows of the cache, each up to its own position. Its keys are blocks
// of 128 positions (aligned, so a page never straddles two blocks). All units' blocks form one
// sequence, each unit's preceded by a few places for what a unit costs beside its blocks (its
// queries, its results), and that is cut into equal runs, one per CTA (one CTA per SM): a run
// takes whole units where they fit and parts of a unit at its ends, so a single long sequence
// and a batch of thousands of short ones both fill the machine, and causal triangles and ragged
// lengths balance by themselves. (Without the places the CTAs with a prompt's first tokens, many
// units of one block, took 1,340 us where the others were done in 560: 3,021 tokens, 64 heads.)
// A part leaves its unnormalised sum, running maximum and sum of weights in the workspace, and a
// second kernel joins the parts. Every CTA finds its run from the lengths on the device: the
// blocks of a sequence's first units are sums of floors, known in closed form.
#pragma once

#include "common.cuh"
#include "paged.h"
#include "waits.cuh"

namespace dsa {
namespace paged {

constexpr int kBlock = 128;        // keys in a block
constexpr int kThreads = 512;      // of both kernels of dsa_paged_attn
constexpr int kMaxCtas = 152;

// Places of a unit before its blocks. (0, 1, 2 and 3 for chunks: 1,534, 1,107, 1,110 and 1,137 us
// for a prompt of 4,096 tokens, 363, 314, 305 and 321 for 34 prompts of 208, 143, 134, 113 and 129
// for 32 users of 64 tokens with a window of 128; for single tokens: 88, 82.5, 83 and 81 us for 64
// users up to 8K.)
constexpr int kUnitCost = 2;

// Softmax. The running maximum m of a row is one of its products s = q . row, unscaled, and a weight
// is exp2((s - m) c), c = scale log2(e): the largest key's is 1 whatever the size of s c. (With
// m = fl(s c) and exp2(fma(s, c, -m)) it is off by 2 to half an ulp of m, a factor that cancels in
// the division by the sum but is zero or infinite from |m| = 2^31 on.)
//
// Two roundings to bf16 are by choice: of the weights and of the rotated dims of the queries, which
// were bf16 when they came in. Both operands of a product have one type, and the rows of the cache
// are bf16; with the weights and rows in tf32 every tile would take twice the shared memory at half
// the rate. The sums of weights take the rounded values, so the weights still add up to one, and
// sums, maxima and outputs stay in fp32 up to the store. An output is off by 0.0018 to 0.0022 of its
// size (2-norm) where rounding it alone gives 0.0017.
constexpr float kRescale = 8.0f;          // log2 units the running maximum may lag behind
constexpr float kNoMax = -3.4028235e38f;  // the maximum of a row that has seen no key: the lowest
                                          // finite value, so that (masked) -inf minus it stays
                                          // -inf and any product replaces it

// Workspace: descriptors, (maximum, sum) of every part's rows, the parts' O. A CTA has two
// slots, as only the first and the last segment of a run can be parts. A slot holds 64 rows of
// 512 dims, row by row, or 128 rows of 256: eight dims (a 32-byte sector) of a row, then the next
// row's, as a thread that holds a row writes them.
constexpr int kMaxRows = 128;
constexpr size_t kSlotFloats = 64 * kD;
constexpr size_t kWsDesc = 0;
constexpr size_t kWsMl = 8192;
constexpr size_t kWsO = kWsMl + size_t{2 * kMaxCtas} * kMaxRows * 2 * sizeof(float);
constexpr size_t kWsAlign = 128;   // the layout begins at the buffer's first multiple of this
static_assert(kWsMl % kWsAlign == 0 && kWsO % kWsAlign == 0, "parts begin lines");
static_assert(kWsO + size_t{2 * kMaxCtas} * kSlotFloats * sizeof(float) + kWsAlign <=
                  DSA_PAGED_WORKSPACE_BYTES,
              "over the workspace");

// Where dim `dim` of row r is in a slot of `rows` rows.
__host__ __device__ constexpr int slot_at(int rows, int r, int dim) {
    return dim / 8 * 8 * rows + r * 8 + dim % 8;
}

// A unit that begins in a CTA's run and ends in a later one, for the join.
struct JoinDesc {
    int64_t row;      // first row of q / out
    int32_t nrows;
    int32_t parts;    // 0: none
    int32_t slot0;    // slot of the first part (the others are slot 0 of the next CTAs)
    int32_t pos;      // position of the unit's first token
    int32_t part;     // which of the group's units
    int32_t pad;
};
static_assert(sizeof(JoinDesc) == 32 && kMaxCtas * sizeof(JoinDesc) <= kWsMl, "descriptors");

struct Params {
    PagedBatch b;
    __nv_bfloat16 *out;
    uint8_t *ws;
    int32_t heads;
    int32_t tpu;       // tokens of a unit
    int32_t upt;       // units of a token group: parts of its heads, or of its output dims
    int32_t rows;      // rows of a unit at most
    int32_t row_step;  // rows from one part's first row to the next part's (0: same rows)
    int32_t rpt;       // rows of a token in a unit
    int32_t window;    // 0: the whole context
    float c;           // scale * log2(e)
    int32_t *status;
    static constexpr bool kSinks = false;
};

// With first tokens that stay visible beside a window. Where a unit's window begins behind block 0,
// they take the first places of the window's first block if these hold keys before the window, whole
// pages of them; otherwise block 0 comes before the window's blocks.
struct SinkParams : Params {
    int32_t sinks;     // 0 without a window; within block 0
    int32_t sink_keys; // keys of their pages, as far as those lie in block 0
    int32_t turn_q;    // q is to be turned by its positions
    static constexpr bool kSinks = true;
};
static_assert(DSA_MAX_SINKS <= kBlock, "the first tokens are in block 0");

// ------------------------------------------------------------------ the list of units
// (each function for both kinds of parameters)

// a / b for a >= 0, b > 0: the 32-bit division where both fit, as they nearly always do.
__device__ __forceinline__ int64_t div_pos(int64_t a, int64_t b) {
    if (((a | b) >> 31) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// sum_{i < n} floor((a + d i) / 128) for a, d >= 0: the whole parts of the slope and the offset in
// closed form, the rest counted along the other axis, where slope and offset are smaller (Graham,
// Knuth and Patashnik, Concrete Mathematics, section 3.5, repeated as in Euclid's algorithm). The
// first step, and the only one of many where d is a power of two, divides by 128.
static __device__ __noinline__ int64_t floor_sum(int64_t n, int64_t a, int64_t d) {
    if (n <= 0) return 0;
    int64_t ans = (n - 1) * n / 2 * (d >> 7) + n * (a >> 7);
    int64_t m = d & 127, y = m * n + (a & 127);
    if (y < kBlock) return ans;
    n = y >> 7;
    a = y & 127;
    d = kBlock;
    for (;;) {
        const int64_t dq = div_pos(d, m), aq = div_pos(a, m);
        ans += (n - 1) * n / 2 * dq + n * aq;
        d -= dq * m;
        a -= aq * m;
        y = d * n + a;
        if (y < m) return ans;
        n = div_pos(y, m);
        a = y - n * m;
        const int64_t t = m;
        m = d;
        d = t;
    }
}

// Keys of the tokens [t0, t1) of a sequence: positions lo .. hi, blocks lo / 128 .. hi / 128.
template <class P>
__device__ __forceinline__ void key_range(const P &p, const PagedSeq &q, int t0, int &lo,
                                          int &hi) {
    const int first = q.len - q.n + t0;
    lo = p.window > 0 ? max(0, first - p.window + 1) : 0;
    hi = q.len - q.n + min(t0 + p.tpu, q.n) - 1;
}

// The number of a unit's first block, its window beginning at lo: that of lo, or one less where the
// first tokens need a block of their own.
template <class P>
__device__ __forceinline__ int first_block(const P &p, int lo) {
    if constexpr (P::kSinks)
        if (lo >= kBlock) lo -= p.sink_keys;
    return lo >> 7;
}

template <class P>
__device__ __forceinline__ int group_blocks(const P &p, const PagedSeq &q, int g) {
    int lo, hi;
    key_range(p, q, g * p.tpu, lo, hi);
    return (hi >> 7) - first_block(p, lo) + 1;
}

// Places of the first G token groups of a sequence, for each part (G = all of them: the last one
// may be short).
template <class P>
static __device__ __noinline__ int64_t places_before_many(const P &p, PagedSeq q, int G) {
    const int base = q.len - q.n, d = p.tpu;
    int64_t sum = floor_sum(G, base + d - 1, d) + int64_t{G} * (1 + kUnitCost);
    if (G * d > q.n) sum += ((q.len - 1) >> 7) - ((base + G * d - 1) >> 7);
    if (p.window > 0) {
        const int a = base - p.window + 1;  // (a window is shorter than the longest sequence)
        // the first group whose window begins at 0 or later; with first tokens, behind block 0
        int first = 0, keys = 0;
        if constexpr (P::kSinks) {
            first = kBlock;
            keys = p.sink_keys;
        }
        const int g0 = a >= first ? 0 : (first - a + d - 1) / d;
        sum -= floor_sum(G - g0, a + g0 * d - keys, d);
    }
    return sum;
}

template <class P>
__device__ __forceinline__ int64_t places_before(const P &p, const PagedSeq &q, int G) {
    return G <= 0 ? 0 : G == 1 ? group_blocks(p, q, 0) + kUnitCost : places_before_many(p, q, G);
}

__device__ __forceinline__ int groups_of(const Params &p, const PagedSeq &q) {
    return (q.n + p.tpu - 1) / p.tpu;
}

__device__ __forceinline__ int64_t unit_row(const Params &p, const PagedSeq &q, int t0, int part) {
    return (int64_t{q.row0} + t0) * p.heads + part * p.row_step;
}

__device__ __forceinline__ int unit_rows(const Params &p, int tokens, int part) {
    return min(p.rows, tokens * p.heads - part * p.row_step);
}

struct Place {
    int s, g, part, off;  // sequence, token group, unit of the group, place of the unit
};

// The token group of a sequence that holds its place r (of all parts' places), by a warp: a round
// looks at 32 groups (a thread that halved 2,048 groups took 35 us of a launch's start).
// Returns it and, above its 32 bits, the place in it.
template <class P>
static __device__ __noinline__ int64_t find_group(const P &p, PagedSeq q, int64_t r) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = groups_of(p, q);  // upt * places_before(lo) <= r < upt * places_before(hi)
    int64_t before = 0;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) >> 5, g = lo + lane * step;
        const int64_t mine = g < hi ? p.upt * places_before(p, q, g) : 0;
        const uint32_t m = __ballot_sync(0xFFFFFFFFu, g < hi && mine <= r) | 1u;
        const int k = 31 - __clz(m);
        before = __shfl_sync(0xFFFFFFFFu, mine, k);
        lo += k * step;
        hi = min(hi, lo + step);
    }
    return (r - before) << 32 | lo;
}

// (all lanes of a warp, with the same arguments)
template <class P>
__device__ __forceinline__ Place find_place(const P &p, const PagedSeq &q, int s, int64_t r) {
    const int64_t at = q.n > p.tpu ? find_group(p, q, r) : r << 32;
    const int g = static_cast<int>(at);
    int in = static_cast<int>(at >> 32), part = 0;
    const int n = group_blocks(p, q, g) + kUnitCost;
    if (in >= n) {  // (upt is 1 or 2)
        in -= n;
        part = 1;
    }
    return Place{s, g, part, in};
}

// Half of the dims (0: dims 0..255) that is the output of a token group's unit `part`, where a
// group has a unit per half. The upper one comes first: its products with new queries begin with
// the dims below 256, which lie in shared memory, and end with those that go through TMEM, which
// arrive last.
__device__ __forceinline__ int half_of(int part) { return part ^ 1; }

// A run of blocks of one unit.
struct Segment {
    int64_t row;       // first row of q / out
    int nrows;         // rows of the unit
    int part;          // which of the group's units
    int s;             // sequence
    int blk;           // first block (positions 128 blk ..)
    int nb;            // blocks
    int posf, posl;    // positions of the unit's first and last token
    int lo;            // lowest position any of its tokens sees
    bool whole;        // all of the unit's blocks
    bool alone;        // the sequence's only unit: nothing else reads its keys
    int ahead;         // keys at the start of the first block that are positions 0 ..; kBlock:
                       // it is block 0, and the next one blk + 1

    // The position of block b, as of its last keys.
    __device__ __forceinline__ int block_pos(int b) const {
        return ahead == kBlock && b == 0 ? 0 : (blk + b) * kBlock;
    }
    // The position of key k of block b.
    __device__ __forceinline__ int key_pos(int b, int k) const {
        return b == 0 && k < ahead ? k : (blk + b) * kBlock + k;
    }
};

// Walks the segments of a CTA's run. Every role walks on its own.
struct Walk {
    Place at;
    PagedSeq q;
    int left;

    template <class P>
    __device__ __forceinline__ Walk(const P &p, const int *start) {
        at = Place{start[0], start[1], start[2], start[3]};
        left = start[4];
        q.n = 0;
        if (left > 0) {
            bool bad;
            q = paged_seq(p.b, at.s, bad);
        }
    }

    template <class P>
    __device__ __forceinline__ bool next(const P &p, Segment &x) {
        if (left <= 0) return false;
        while (at.g * p.tpu >= q.n) {
            if (++at.s >= p.b.n_seqs) return false;
            at.g = 0;
            bool bad;
            q = paged_seq(p.b, at.s, bad);
        }
        const int t0 = at.g * p.tpu, t1 = min(t0 + p.tpu, q.n);
        int hi;
        key_range(p, q, t0, x.lo, hi);
        const int blo = first_block(p, x.lo), nblk = (hi >> 7) - blo + 1;
        const int before = max(0, kUnitCost - at.off), off = max(0, at.off - kUnitCost);
        x.nb = min(nblk - off, left - before);
        if (x.nb <= 0) {  // the run ends before the unit's first block
            left = 0;
            return false;
        }
        x.s = at.s;
        x.posf = q.len - q.n + t0;
        x.posl = hi;
        x.row = unit_row(p, q, t0, at.part);
        x.nrows = unit_rows(p, t1 - t0, at.part);
        x.part = at.part;
        x.blk = blo + off;
        x.ahead = 0;
        if constexpr (P::kSinks)
            if (off == 0 && x.lo >= kBlock) x.ahead = blo < x.lo >> 7 ? kBlock : p.sink_keys;
        x.whole = x.nb == nblk;
        x.alone = p.upt == 1 && q.n <= p.tpu;
        left -= before + x.nb;
        at.off = 0;
        if (++at.part == p.upt) {
            at.part = 0;
            ++at.g;
        }
        return true;
    }
};

// Walks a run block by block for the loaders: the lane's page of each block, ahead of its load.
struct PageWalk {
    Walk walk;
    Segment x;
    int b;
    bool have;

    template <class P>
    __device__ __forceinline__ PageWalk(const P &p, const int *start) : walk(p, start), b(0) {
        have = walk.next(p, x);
    }

    // The page that holds this lane's rows [pos, pos + prows) of the next block (-1: no token
    // needs one, or a bad table entry), and the row of the page they begin at.
    template <class P>
    __device__ __forceinline__ int32_t next(const P &p, int page, int prows, int pages,
                                            int &row) {
        int32_t e = -1;
        if (have) {
            const int pos = x.key_pos(b, page * prows);
            row = pos & ((1 << p.b.page_shift) - 1);
            bool seen = pos > x.lo - prows;
            if constexpr (P::kSinks) seen |= pos < p.sinks;
            if (page < pages && pos <= x.posl && seen) {
                e = __ldg(p.b.page_table + int64_t{x.s} * p.b.max_pages + (pos >> p.b.page_shift));
                if (e < 0 || e >= p.b.n_pages) {
                    report(p.status, DSA_ERR_BOUNDS);
                    e = -1;
                }
            }
            if (++b == x.nb) {
                b = 0;
                have = walk.next(p, x);
            }
        }
        return e;
    }
};

// Position of row r of a unit.
__device__ __forceinline__ int row_pos(const Params &p, int posf, int r) {
    return p.tpu == 1 ? posf : posf + r / p.rpt;
}

// Finds this CTA's run, places [T0, T1) of all places: start[0..3] its first place, start[4] its
// length (0 on entry); describes the unit that begins in it and ends beyond for the join. All
// threads call it; `scratch` holds a value per warp and four more. Ends with a barrier of the CTA,
// and one inside it publishes what was set up before (TMEM, mbarriers).
template <int kT = kThreads, class P>
__device__ __forceinline__ void find_run(const P &p, int64_t *scratch, int *start) {
    constexpr int kWarps = kT / 32;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = static_cast<int>(blockIdx.x);
    JoinDesc *desc = reinterpret_cast<JoinDesc *>(p.ws + kWsDesc) + cta;
    const int per = (p.b.n_seqs + kT - 1) / kT;
    const int s0 = min(tid * per, p.b.n_seqs), s1 = min(s0 + per, p.b.n_seqs);
    int64_t mine = 0, nb = 0;
    PagedSeq q = {};
    for (int s = s0; s < s1; ++s) {
        bool bad;
        q = paged_seq(p.b, s, bad);
        if (bad && cta == 0) report(p.status, DSA_ERR_BOUNDS);
        nb = p.upt * places_before(p, q, groups_of(p, q));
        mine += nb;
    }
    int64_t incl = mine;
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, incl, w);
        if (lane >= w) incl += v;
    }
    if (lane == 31) scratch[warp] = incl;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // (scanned once more in every warp; few instructions, as each is fetched cold)
    int64_t upto = lane < kWarps ? scratch[lane] : 0;
#pragma unroll
    for (int w = 1; w < kWarps; w <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, upto, w);
        if (lane >= w) upto += v;
    }
    const int64_t total = __shfl_sync(0xFFFFFFFFu, upto, kWarps - 1);
    const int64_t below = __shfl_sync(0xFFFFFFFFu, upto, warp > 0 ? warp - 1 : 0);
    if (warp > 0) incl += below;
    const int64_t run = div_pos(total + gridDim.x - 1, gridDim.x);
    const int64_t T0 = run * cta, T1 = min(T0 + run, total);
    int64_t *const ends = scratch + kWarps;  // sequence and place in it: the run's first
                                                    // place, its last
    if (mine > 0 && T0 < T1 && T0 < incl && T1 > incl - mine) {
        // one of this thread's sequences holds the first, the last, or both
        int64_t acc = incl - mine;
        for (int s = s0; s < s1; ++s) {
            if (s1 - s0 > 1) {
                bool bad;
                q = paged_seq(p.b, s, bad);
                nb = p.upt * places_before(p, q, groups_of(p, q));
            }
            if (T0 >= acc && T0 < acc + nb) {
                ends[0] = s;
                ends[1] = T0 - acc;
            }
            if (T1 > acc && T1 <= acc + nb) {
                ends[2] = s;
                ends[3] = T1 - 1 - acc;
            }
            acc += nb;
        }
    }
    __syncthreads();
    if (T0 >= T1) {
        if (tid == 0) *desc = JoinDesc{};
    } else if (warp < 2) {
        const int s = static_cast<int>(ends[2 * warp]);
        bool bad;
        q = paged_seq(p.b, s, bad);
        const Place x = find_place(p, q, s, ends[2 * warp + 1]);
        if (warp == 0 && lane == 0) {
            start[0] = x.s;
            start[1] = x.g;
            start[2] = x.part;
            start[3] = x.off;
            start[4] = static_cast<int>(T1 - T0);
        }
        if (warp == 1 && lane == 0) {
            // the unit of the last place: does its first block lie in this run, and its last one
            // in a later run?
            const int64_t u0 = T1 - 1 - x.off;
            const int64_t u1 = u0 + kUnitCost + group_blocks(p, q, x.g);
            JoinDesc d = {};
            if (x.off >= kUnitCost && u0 + kUnitCost >= T0 && u1 > T1) {
                const int t0 = x.g * p.tpu, t1 = min(t0 + p.tpu, q.n);
                d.row = unit_row(p, q, t0, x.part);
                d.nrows = unit_rows(p, t1 - t0, x.part);
                d.part = x.part;
                d.parts = static_cast<int>(div_pos(u1 - 1, run)) - cta + 1;
                d.slot0 = u0 <= T0 ? 0 : 1;
                d.pos = q.len - q.n + t0;
            }
            *desc = d;
        }
    }
    fence_proxy_async_smem();  // the scratch's tile is next written by TMA
    __syncthreads();
}

// ------------------------------------------------------------------ small helpers

__device__ __forceinline__ float redux_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint64_t policy_evict_normal() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *tm, uint64_t *bar, int x,
                                            int y, int z, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
        "l"(tm), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}

__device__ __forceinline__ void prefetch_tmap(const CUtensorMap *tm) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(tm) : "memory");
}

// mbar_wait whose loop is out of line and whose budget counts from the last block.
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, volatile int *abort,
                                         int32_t *status) {
    return mbar_test(smem_u32(bar), parity) || wait_moving(bar, parity, abort, status);
}

// One lane of a converged warp, the same one every time. A branch on it (rather than on
// lane == 0) lets the compiler keep what the tensor instructions take in uniform registers:
// M=128 N=16 MMAs issue one per 39 cycles behind it, one per 59 behind lane == 0, one per 81
// from a converged warp with a predicate (the products here need one per 48 to 64).
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.b32 %0, 1, 0, p;\n}\n"
        : "=r"(r));
    return r != 0;
}

__device__ __forceinline__ void drain_wait(uint64_t *bar, uint32_t parity) {
    const uint32_t b = smem_u32(bar);
    const long long t0 = clock64();
    while (!mbar_test(b, parity))
        if (clock64() - t0 > kWaitBudget) break;
}

// Two floats as the operand of an instruction that works on both (fewer instructions in the
// softmax: a 2,048-token chunk at 16K 3,790 -> 3,650 us, a window of 128 209 -> 202).
__device__ __forceinline__ uint64_t pair_of(uint32_t lo, uint32_t hi) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(lo), "r"(hi));
    return v;
}

__device__ __forceinline__ uint64_t pair_of(float both) {
    return pair_of(__float_as_uint(both), __float_as_uint(both));
}

__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t v;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
    return v;
}

__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
    uint64_t v;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}

__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
    uint64_t v;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}

__device__ __forceinline__ float first_of(uint64_t v) {
    return __uint_as_float(static_cast<uint32_t>(v));
}

__device__ __forceinline__ float second_of(uint64_t v) {
    return __uint_as_float(static_cast<uint32_t>(v >> 32));
}

// Both bf16 values of a word with infinities and NaN replaced by zero.
__device__ __forceinline__ uint32_t finite2(uint32_t v) {
    if ((v & 0x7F800000u) == 0x7F800000u) v &= 0x0000FFFFu;
    if ((v & 0x00007F80u) == 0x00007F80u) v &= 0xFFFF0000u;
    return v;
}

}  // namespace paged

// The chunk kernel (paged_chunk.cu): one-time set-up, and its launch.
constexpr int kChunkRows = 128;
int prepare_paged_chunk();

// The join of the units that paged_attn_kernel (or one that leaves the same parts) cut.
int enqueue_paged_join(const paged::Params &p, int ctas, cudaStream_t s);

// Places that a CTA's run may have (of a GB300's 152), from the sizes alone (lengths are the
// device's): the kernels count them in 32 bits. `keys`: the longest range of a unit's keys.
int64_t paged_run_bound(const paged::Params &p, int64_t keys);

int enqueue_paged_chunk(const CUtensorMap &tm_q, const CUtensorMap &tm_kv,
                        const paged::Params &p, const void *q, int ctas, cudaStream_t s);

}  // namespace dsa
