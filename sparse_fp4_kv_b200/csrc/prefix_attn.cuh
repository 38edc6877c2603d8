// prefix_attn.cuh -- decode attention for sequences that share a prefix.
//
// Sequences come in groups; entries below a group's prefix length are read
// through the pages of the group's first member, later ones through the
// sequence's own pages, and each query's window rows are attended too:
//     o_h = sum_j softmax_j(scale * <q_h, v_j>) v_j
// over the entries below the query's limit and its window rows (each row is
// key and value, as in attn_decode.cuh).
//
// Bound. A prefix entry (288 bytes) meets every (query, head) row of its
// group: 4 * 512 flops per row and entry, so from about 100 rows on the
// tensor pipe bounds the prefix, not memory. The work is therefore cut by
// rows, not by sequences: a strip is up to 128 rows of one group against the
// group's prefix, or the heads of one query against its own rows (the entries
// behind the prefix, then its window). A strip's rows of the cache are cut
// into tiles of 256; all tiles form one list, and every pair of CTAs takes an
// equal share of it. A share's part of a strip leaves an f32 partial (o divided
// by its own denominator, and its log-sum-exp); k_prefix_merge joins a
// query's partials of its prefix strip and of its own.
//
// Tile. A pair of CTAs (cta_group::2, M = 128: 64 rows of the strip each)
// holds O [128][512] in f32 in both TMEMs: each CTA keeps its 64 rows, the
// lanes 0..63 columns 0..255 and the lanes 64..127 columns 256..511. For S a
// CTA holds the keys of half of the tile (128 of the N = 256 columns), for
// P V all 256 rows of half of the latent width. One CTA alone could not:
// O of 128 rows fills its TMEM, and of 64 rows costs the tensor pipe as much
// as 128. N = 256 for both products: an instruction reads 6 KiB of operands from
// shared memory in its 64 cycles (N = 128: 4 KiB in 32), which leaves room for
// the stores of dequantised rows.
// Shared memory: Q (64 KiB), P (32 KiB) and a ring of four 32 KiB chunks, in
// the order the products take them: four chunks of 128 latent values of the
// keys of tile i + 1, then up to four chunks of 64 rows of the values of
// tile i, so that S of the next tile runs while the softmax of a tile does.
//
// Warps: 4 of softmax (a thread has half a row: 128 scores), 16 that fetch rows
// into registers a group of chunks ahead, dequantise them (exact in f16) and
// store them, one that issues the products (in the first CTA), one that resolves
// rows up to four tiles ahead, one that has q copied in.
//
// Measured (8 queries x 64 heads on 200,000 shared entries: 3128 tiles): 195 us,
// 1.08 PFLOP/s. A tile takes 7300 cycles, 4096 of them the tensor pipe's (55 %
// active); the array of L1 and shared memory is busy 73 % with loads and stores,
// beside the products' operands. At 1000 W the clock falls to 1.5 - 1.6 GHz, so
// what is left to gain is work that is not done rather than waits.
#pragma once

#include "common.cuh"

namespace csa2 {

// One strip: rows of queries against a list of cache rows.
struct __align__(16) PrefixStrip {
    int64_t tile0;     // first tile in the call's list
    int64_t cost0;     // the same in the list's costs (see px_lo)
    int32_t ntiles;    // tiles of 256 rows (0: nothing to attend)
    int32_t rows;      // length of the list of cache rows
    int32_t seq;       // page-table row of its entries
    int32_t t_base;    // id of the first entry
    int32_t entries;   // FP4 entries of the list; the rest are window rows
    int32_t w_begin;   // ring slot of the first window row
    int32_t q_rows;    // rows of queries, at most 128
    int32_t member0;   // prefix: first member of the group; own: -1
    int32_t row0;      // prefix: first row among the group's (member, query, head) rows; own: 0
    int32_t q_at;      // first row in q16
    int32_t w_seq;     // sequence of the window
};

// What the merge has to know of one query: where the partials of its rows are.
struct __align__(16) PrefixItem {
    int64_t pre_cost0, own_cost0;  // cost0 of its group's first strip, of its own strip
    int32_t pre_strip, pre_tiles;  // first strip of the group, tiles of each (0: none)
    int32_t x0;                    // its first row among the group's rows
    int32_t own_tiles;
    int32_t u;                     // its number, -1: not computed
    int32_t group;
};

struct PrefixParams {
    const uint16_t *q;  // bf16 [nq][h][512]
    csa2_kv_desc kv;
    const int32_t *members, *group_begin, *prefix_len;
    const int32_t *q_limit;  // nullable
    const uint8_t *swa;      // nullable, with begin / end
    int64_t swa_seq_stride;
    const int32_t *swa_begin, *swa_end;
    uint16_t *o;
    float *lse;        // nullable
    float scale_log2;  // |softmax scale| * log2(e), above 0
    uint32_t q_flip;   // sign bits of two f16 values when the softmax scale is negative
    int32_t nq, q_per_seq, h, w_max, n_members, n_groups, pairs;
    // workspace
    int64_t *total_tiles;   // [2] tiles, and their cost with the strips'
    int32_t *n_pre;         // [1] prefix strips
    int32_t *start;         // [pairs] first strip of each pair's run
    int64_t *start_tile;    // [pairs + 1] first tile of each run
    PrefixItem *items;      // [n_members * q_per_seq]
    // of each group, when there are more than kPxPlanGroups (else in shared memory):
    // entries of the prefix that any query sees, first strip, its cost0, tiles
    int32_t *group_seen, *group_strip, *group_tiles;
    int64_t *group_cost;
    PrefixStrip *strips;    // [max_pre + n_members * q_per_seq], the prefix strips first
    int32_t max_pre;
    uint16_t *q16;          // [n_members * q_per_seq * h][512] q in f16, in the order of members
    float *pre_o, *pre_lse;  // [pairs + max_pre][128][512], [..][128]
    float *own_o, *own_lse;  // [pairs + n_members * q_per_seq][h][512], [..][h]
};

constexpr int kPxTile = 256;  // cache rows of a tile
constexpr int kPxRows = 128;  // query rows of a strip
constexpr int kPxSoftWarps = 4;
constexpr int kPxLoadWarps = 16;
constexpr int kPxMmaWarp = kPxSoftWarps + kPxLoadWarps;
constexpr int kPxThreads = (kPxMmaWarp + 4) * 32;  // products, resolver, q, and one idle warp
constexpr int kPxSlots = 4;
constexpr int kPxSlotBytes = 32768;
constexpr int kPxQBytes = 64 * CSA2_D * 2;
constexpr int kPxPBytes = 64 * kPxTile * 2;
constexpr int kPxMisc = 2048;
constexpr size_t kPxSmem = 1024 + kPxQBytes + kPxPBytes + (size_t)kPxSlots * kPxSlotBytes + kPxMisc;
constexpr float kPxRescale = 8.0f;  // log2 by which the maximum may rise before O is rescaled
// Probabilities are f16 (11 bits, which is what the products take), but their sum
// is f32. In a long list many small ones may weigh more than f16's least number
// lets through, so they are taken 2^kPxBias times as large: at most 2^15, and one
// is rounded by at most 2^-32 of the largest (2^-25 without; a million entries at
// 2^-25.5 of one lost 2 % of the result).
constexpr float kPxBias = 7.0f;
static_assert(kPxRescale + kPxBias <= 15.0f, "probabilities stay finite in f16");
static_assert(kPxSmem <= 232448, "shared memory of one CTA");
static_assert(kPxSlots == 4 && kPxLoadWarps == 4 * kPxSlots, "a set of four warps a slot");

// ---------------------------------------------------------------------------
// cta_group::2 forms and cluster-scope barriers
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tmem_alloc2(uint32_t *dst, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(ncols)
                 : "memory");
}
__device__ __forceinline__ void tmem_relinquish2() {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc2(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void mma_f16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrives on the same barrier of both CTAs when the products issued so far are done.
__device__ __forceinline__ void tc_commit_pair(uint64_t *bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}
// Arrives at a barrier of either CTA of the pair. Scope CTA (the default) on
// purpose: what these barriers announce lies in the arriving CTA's own shared
// memory, written there and fenced for the async proxy before, and is read by
// that CTA's tensor core. Releasing at cluster scope took 930 cycles in a warp
// with loads in flight and bounded the kernel (12,000 cycles a tile).
__device__ __forceinline__ void mbar_arrive_pair(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// Registers of the calling group of four warps. The six groups' shares sum up to
// what the block is launched with (6 x 80): softmax 152, rows 4 x 72, products
// 40. None spills: a spill is a trip to L2, as the carve-out for shared memory
// leaves little L1.
template <int N>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t yes;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
    return yes != 0;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ---------------------------------------------------------------------------
// the split of the tile list over the pairs: equal shares of a cost of one per
// tile and kPxStripCost per strip (loading its q, filling the pipeline and
// storing its partial). No more pairs than the cost, so that a strip's partials
// are those of consecutive pairs.
// ---------------------------------------------------------------------------
constexpr int kPxStripCost = 2;
__device__ __forceinline__ int32_t px_pairs(int32_t pairs, int64_t cost) { return (int32_t)min((int64_t)pairs, cost); }
__device__ __forceinline__ int64_t px_lo(int64_t cost, int32_t pairs, int64_t c) { return c * cost / pairs; }
// the pair whose share holds tile x of the strip that begins at cost0
__device__ __forceinline__ int32_t px_owner(int64_t cost, int32_t pairs, int64_t cost0, int32_t x) {
    return (int32_t)(((cost0 + kPxStripCost + x + 1) * pairs - 1) / cost);
}

// Visible entries of query u of sequence s: at most what a row of the page table
// holds and 2^30, so that a list of entries and window rows stays below 2^31.
constexpr int32_t kPxMostRows = 1 << 30;
__device__ __forceinline__ int32_t px_limit(const PrefixParams &p, int32_t s, int64_t u) {
    const int64_t room = min((int64_t)p.kv.max_pages * p.kv.page_size, (int64_t)kPxMostRows);
    const int32_t n = p.q_limit ? p.q_limit[u] : p.kv.seq_len[s];
    if (n > room) set_error(CSA2_DEVERR_BAD_ROW);
    return (int32_t)min((int64_t)max(n, 0), room);
}

// ---------------------------------------------------------------------------
// plan: one block lists the strips. Its time is that of its dependent loads and
// barriers, so threads keep what they computed (one query and one strip each, up
// to 1024) and the groups' numbers stay in shared memory.
// ---------------------------------------------------------------------------
constexpr int kPxPlanThreads = 1024;
constexpr int kPxPlanGroups = 1024;

// Exclusive sums of two values over the block, and their totals.
__device__ __forceinline__ void px_block_exclusive(int64_t (&v)[2], int64_t (*sums)[32], int64_t (&total)[2]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t s[2] = {v[0], v[1]};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int64_t u = __shfl_up_sync(0xFFFFFFFFu, s[k], o);
            if (lane >= o) s[k] += u;
        }
    if (lane == 31) sums[0][warp] = s[0], sums[1][warp] = s[1];
    __syncthreads();
    if (warp < 2) {
        int64_t w = sums[warp][lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xFFFFFFFFu, w, o);
            if (lane >= o) w += u;
        }
        sums[warp][lane] = w;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        v[k] = (warp ? sums[k][warp - 1] : 0) + s[k] - v[k];
        total[k] = sums[k][31];
    }
    __syncthreads();
}
static_assert(kPxPlanThreads == 1024, "px_block_exclusive sums 32 warps");

// The last k in [0, n) with a[k] <= x of an ascending list; -1: none.
__device__ __forceinline__ int32_t px_last_below(const int32_t *a, int32_t n, int32_t x) {
    int32_t lo = 0, hi = n;  // a[k] <= x for k < lo, > x for k >= hi
    while (lo < hi) {
        const int32_t m = (lo + hi) >> 1;
        if (a[m] <= x) lo = m + 1;
        else hi = m;
    }
    return lo - 1;
}

// q in f16 (the sign turned for a negative scale), rows in the order of members:
// the rows of a strip then lie together and one tiled copy a block of 64
// positions brings them into shared memory, swizzled. The latent values stand in
// the order that the cache's rows get (PxRaw). 16 bytes a thread.
__device__ __forceinline__ void px_convert_q(const PrefixParams &p, int64_t rows) {
    const int64_t step = (int64_t)(gridDim.x - 1) * kPxPlanThreads;
    bool bad = false;
    for (int64_t i = (int64_t)(blockIdx.x - 1) * kPxPlanThreads + threadIdx.x; i < rows * (CSA2_D / 8); i += step) {
        const int32_t row = (int32_t)(i / (CSA2_D / 8)), c = (int32_t)(i % (CSA2_D / 8));
        const int32_t per = p.q_per_seq * p.h, j = row / per, y = row - j * per;
        const int32_t seq = p.members[j];
        uint32_t w[4] = {0u, 0u, 0u, 0u};
        if (seq >= 0 && seq < p.kv.batch) {
            const int64_t u = (int64_t)seq * p.q_per_seq + y / p.h;
            if (u < p.nq) {
                // piece m of a 128: pairs 32 q + 2 m
                const uint32_t *at = reinterpret_cast<const uint32_t *>(p.q + (u * p.h + y % p.h) * CSA2_D) + (c >> 4) * 64 + (c & 15);
#pragma unroll
                for (int k = 0; k < 4; ++k) w[k] = __ldg(at + 16 * k);
            }
        }
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            // 65536 and more (0x4780 and up, infinities and NaN too) have no finite f16 value
            bad |= (w[k] & 0x7FFFu) >= 0x4780u || ((w[k] >> 16) & 0x7FFFu) >= 0x4780u;
            const __half2 h = __floats2half2_rn(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u));
            o[k] = *reinterpret_cast<const uint32_t *>(&h) ^ p.q_flip;
        }
        reinterpret_cast<uint4 *>(p.q16)[i] = make_uint4(o[0], o[1], o[2], o[3]);
    }
    if (bad) set_error(CSA2_DEVERR_Q_RANGE);
}

// Notes the pairs whose share of the cost begins in strip i.
__device__ __forceinline__ void px_note_starts(const PrefixParams &p, int32_t i, int64_t tile0, int64_t cost0, int32_t ntiles, int64_t cost,
                                               int32_t pairs) {
    if (ntiles == 0) return;
    // pairs c with cost0 <= lo(c) < cost0 + kPxStripCost + ntiles
    const int64_t end = cost0 + kPxStripCost + ntiles;
    for (int64_t c = (cost0 * pairs + cost - 1) / cost; c < pairs && px_lo(cost, pairs, c) < end; ++c) {
        p.start[c] = i;
        p.start_tile[c] = tile0 + max((int64_t)0, px_lo(cost, pairs, c) - cost0 - kPxStripCost);
    }
}

__global__ void __launch_bounds__(kPxPlanThreads) k_prefix_plan(PrefixParams p) {
    __shared__ int64_t sums[2][32];
    __shared__ int32_t descends;
    __shared__ int32_t begin_s[kPxPlanGroups + 1], seen_s[kPxPlanGroups], strip_s[kPxPlanGroups], tiles_s[kPxPlanGroups];
    __shared__ int64_t cost_s[kPxPlanGroups];
    const int tid = threadIdx.x;
    pdl_trigger();
    pdl_wait();
    const int32_t n_own = p.n_members * p.q_per_seq, per = p.q_per_seq * p.h;
    if (blockIdx.x > 0) {
        px_convert_q(p, (int64_t)n_own * p.h);
        return;
    }
    const bool few = p.n_groups <= kPxPlanGroups;
    const int32_t *begin = few ? begin_s : p.group_begin;
    // volatile: raised by atomics, which a line in L1 would not show
    volatile int32_t *seen = few ? seen_s : p.group_seen;
    int32_t *g_strip = few ? strip_s : p.group_strip, *g_tiles = few ? tiles_s : p.group_tiles;
    int64_t *g_cost = few ? cost_s : p.group_cost;
    if (tid == 0) descends = 0;
    __syncthreads();
    for (int32_t g = tid; g < p.n_groups; g += kPxPlanThreads) {
        const int32_t b0 = p.group_begin[g], b1 = p.group_begin[g + 1];
        if (b0 > b1) descends = 1;
        if (b0 < 0 || b1 > p.n_members) set_error(CSA2_DEVERR_BAD_ROW);
        if (few) {
            begin_s[g] = b0;
            if (g == p.n_groups - 1) begin_s[g + 1] = b1;
        }
        seen[g] = 0;
    }
    __syncthreads();
    // groups that overlap could not be told apart: a list that descends is refused as a whole
    const bool all_bad = descends != 0;
    if (all_bad && tid == 0) set_error(CSA2_DEVERR_BAD_ROW);
    PrefixStrip *own = p.strips + p.max_pre;
    // ---- each query's own list, and how much of the prefix it sees ----
    int32_t my_tiles = 0;        // of the thread's first query
    PrefixItem my_item;
    my_item.u = -1;
    for (int32_t i = tid; i < n_own; i += kPxPlanThreads) {
        const int32_t j = i / p.q_per_seq, qi = i - j * p.q_per_seq;
        const int32_t s = p.members[j];
        const int64_t u = (int64_t)s * p.q_per_seq + qi;
        const bool there = s >= 0 && s < p.kv.batch;
        if (!there) set_error(CSA2_DEVERR_BAD_ROW);
        int32_t limit = 0, wb = 0, nw = 0;
        if (there && u < p.nq) {
            limit = px_limit(p, s, u);
            if (p.swa_begin) {
                wb = p.swa_begin[u];
                nw = max(0, p.swa_end[u] - wb);
            }
        }
        const int32_t g = all_bad ? -1 : px_last_below(begin, p.n_groups + 1, j);
        PrefixItem item;
        item.u = -1;
        item.group = -1;
        item.own_tiles = 0;
        if (there && u < p.nq && g >= 0 && g < p.n_groups && begin[g] >= 0 && begin[g + 1] <= p.n_members) {
            const int32_t prefix = max(0, p.prefix_len[g]), b0 = begin[g], head = p.members[b0];
            if (head >= 0 && head < p.kv.batch && min(limit, prefix) > 0) atomicMax(const_cast<int32_t *>(seen) + g, min(limit, prefix));
            if (nw > 0 && (wb < 0 || wb >= p.swa_seq_stride || nw > p.swa_seq_stride || nw > p.w_max)) {
                set_error(CSA2_DEVERR_BAD_ROW);
                nw = 0;
            }
            PrefixStrip t;
            t.tile0 = t.cost0 = 0;
            t.entries = max(0, limit - prefix);
            t.rows = t.entries + nw;
            t.ntiles = (t.rows + kPxTile - 1) / kPxTile;
            t.seq = s;
            t.t_base = prefix;
            t.w_begin = wb;
            t.q_rows = p.h;
            t.member0 = -1;
            t.row0 = 0;
            t.q_at = i * p.h;
            t.w_seq = s;
            own[i] = t;
            item.u = (int32_t)u;
            item.group = g;
            item.x0 = (j - b0) * per + qi * p.h;
            item.own_tiles = t.ntiles;
        } else {
            own[i].ntiles = 0;
        }
        if (i == tid) {
            my_tiles = item.own_tiles;
            my_item = item;
        } else {
            p.items[i] = item;
        }
    }
    __syncthreads();
    // ---- the groups' strips ----
    int64_t strips = 0, tiles = 0;
    for (int32_t g0 = 0; g0 < p.n_groups; g0 += kPxPlanThreads) {
        const int32_t g = g0 + tid;
        int32_t n = 0, nt = 0;
        if (g < p.n_groups && seen[g] > 0) {
            n = ((begin[g + 1] - begin[g]) * per + kPxRows - 1) / kPxRows;
            nt = (seen[g] + kPxTile - 1) / kPxTile;
        }
        int64_t v[2] = {n, (int64_t)n * nt}, t[2];
        px_block_exclusive(v, sums, t);
        if (g < p.n_groups) {
            g_strip[g] = (int32_t)(strips + v[0]);
            g_tiles[g] = nt;
            g_cost[g] = tiles + v[1] + kPxStripCost * (strips + v[0]);  // every prefix strip has tiles
        }
        strips += t[0];
        tiles += t[1];
    }
    const int32_t n_pre = (int32_t)min(strips, (int64_t)p.max_pre);
    __syncthreads();
    int64_t cost = tiles + kPxStripCost * strips;
    // ---- where each query's own strip lies ----
    int64_t my_tile0 = 0, my_cost0 = 0;
    for (int32_t i0 = 0; i0 < n_own; i0 += kPxPlanThreads) {
        const int32_t i = i0 + tid;
        PrefixItem item = my_item;
        if (i0 > 0 && i < n_own) item = p.items[i];
        const int32_t nt = i < n_own ? item.own_tiles : 0;
        int64_t v[2] = {nt, nt ? nt + kPxStripCost : 0}, t[2];
        px_block_exclusive(v, sums, t);
        if (i < n_own) {
            own[i].tile0 = tiles + v[0];
            own[i].cost0 = cost + v[1];
            item.own_cost0 = cost + v[1];
            if (item.group >= 0) {
                item.pre_strip = g_strip[item.group];
                item.pre_tiles = g_tiles[item.group];
                item.pre_cost0 = g_cost[item.group];
            }
            p.items[i] = item;
            if (i0 == 0) my_tile0 = tiles + v[0], my_cost0 = cost + v[1];
        }
        tiles += t[0];
        cost += t[1];
    }
    const int32_t pairs = px_pairs(p.pairs, cost);
    if (tid == 0) {
        p.total_tiles[0] = tiles;
        p.total_tiles[1] = cost;
        *p.n_pre = n_pre;
        p.start_tile[pairs] = tiles;
    }
    if (tiles == 0) return;
    // ---- the prefix strips, and where each pair's share begins ----
    for (int32_t s = tid; s < n_pre; s += kPxPlanThreads) {
        const int32_t g = px_last_below(g_strip, p.n_groups, s);  // of equal ones the last: the group that has strips
        const int32_t x = s - g_strip[g], b0 = begin[g], rows = (begin[g + 1] - b0) * per;
        PrefixStrip t;
        t.ntiles = g_tiles[g];
        t.cost0 = g_cost[g] + (int64_t)x * (t.ntiles + kPxStripCost);
        t.tile0 = t.cost0 - (int64_t)kPxStripCost * s;
        t.rows = t.entries = seen[g];
        t.seq = p.members[b0];
        t.t_base = 0;
        t.w_begin = 0;
        t.q_rows = min(kPxRows, rows - x * kPxRows);
        t.member0 = b0;
        t.row0 = x * kPxRows;
        t.q_at = b0 * per + x * kPxRows;
        t.w_seq = 0;
        p.strips[s] = t;
        px_note_starts(p, s, t.tile0, t.cost0, t.ntiles, cost, pairs);
    }
    for (int32_t i = tid; i < n_own; i += kPxPlanThreads) {
        if (i == tid) px_note_starts(p, n_pre + i, my_tile0, my_cost0, my_tiles, cost, pairs);
        else px_note_starts(p, n_pre + i, own[i].tile0, own[i].cost0, own[i].ntiles, cost, pairs);
    }
}

// A role's walk over the tiles of a pair's run.
struct PxWalk {
    PrefixStrip t;
    int32_t s, tile, n_pre;  // strip, tile within it
    __device__ __forceinline__ void load(const PrefixParams &p) {
        t = s < n_pre ? p.strips[s] : p.strips[p.max_pre + (s - n_pre)];
    }
    __device__ __forceinline__ void begin(const PrefixParams &p, int32_t c, int64_t x0) {
        n_pre = *p.n_pre;
        s = p.start[c];
        load(p);
        tile = (int32_t)(x0 - t.tile0);
    }
    __device__ __forceinline__ bool last() const { return tile == t.ntiles - 1; }
    // only while tiles are left: strips without tiles are passed over
    __device__ __forceinline__ void next(const PrefixParams &p) {
        if (++tile < t.ntiles) return;
        tile = 0;
        do {
            ++s;
            load(p);
        } while (t.ntiles == 0);
    }
    __device__ __forceinline__ int value_chunks() const { return (min(kPxTile, t.rows - tile * kPxTile) + 63) >> 6; }
};

// Where a row of a tile lies: >= 0 a physical cache row, kPxNone no row, else
// -2 - slot of the window ring. Resolved in two steps, so that the page-table
// load is in flight while a group of chunks is handled: px_look gives, for an
// entry, the row within its page and starts the load of the page number.
constexpr int32_t kPxNone = -1;
struct PxLook {
    int32_t code, page;
};
template <class T>  // a strip or what an info tells of one
__device__ __forceinline__ void px_look(const PrefixParams &p, const T &strip, int32_t tile, int r, PxLook &x) {
    const int32_t j = tile * kPxTile + r;
    x.code = kPxNone;
    x.page = -1;
    if (j < strip.entries) {
        const uint32_t t = (uint32_t)strip.t_base + (uint32_t)j;  // below max_pages * page_size (px_limit)
        const uint32_t page = t / (uint32_t)p.kv.page_size;
        x.code = (int32_t)(t - page * (uint32_t)p.kv.page_size);
        x.page = p.kv.page_table[(int64_t)strip.seq * p.kv.max_pages + page];
    } else if (j < strip.rows) {
        int64_t sl = (int64_t)strip.w_begin + (j - strip.entries);  // below twice the stride
        if (sl >= p.swa_seq_stride) sl -= p.swa_seq_stride;
        x.code = -2 - (int32_t)sl;
    }
}
__device__ __forceinline__ int32_t px_row(const PrefixParams &p, const PxLook &x) {
    if (x.code < 0) return x.code;
    const int64_t row = (int64_t)x.page * p.kv.page_size + x.code;
    if (x.page >= 0 && row < p.kv.rows_cap) return (int32_t)row;
    set_error(CSA2_DEVERR_BAD_ROW);
    return kPxNone;
}

// What a CTA's resolver warp tells of a tile, up to kPxInfos tiles ahead. Its 256
// rows are 16 runs of 16: base[g] is the cache row of the run's first row when
// the run is 16 entries of one page, kPxWindow - slot when it is 16 rows of the
// window ring from that slot on, kPxNone when it holds no row at all, and
// kPxMixed otherwise (a run across pages, cut off, both entries and window, or
// with bad pages: the warps that fetch it resolve its rows themselves).
constexpr int kPxInfos = 4;
constexpr int32_t kPxMixed = -2, kPxWindow = -3;
struct __align__(16) PxInfo {
    int32_t base[16];
    uint32_t valid[8];  // rows there are, a bit each
    int32_t tile, left;
    int32_t seq, t_base, entries, rows, w_begin, w_seq;  // as in the strip
};

// A lane's share of a chunk: four units of 32 consecutive values of a row (16
// bytes of codes and 2 of scales, or 32 bytes of a window row). A warp's unit is
// eight rows of 128 values, four lanes a row, so that its loads take whole
// 64-byte runs (lanes with a row each touched 32 lines a load, which made the L1
// array the bound), and its stores are 8 x 8 matrices: lane 4 r + q holds the
// pair of values that stmatrix puts at columns 2 q, 2 q + 1 of row r. To need no
// exchange between lanes, the latent values of each 128 are taken in the order
//     position 8 m + 2 q + e  <-  value 32 q + 2 m + e   (m < 16, q < 4, e < 2),
// pair m of lane q's unit being what it stores to matrix m. The products do not
// mind an order of the latent axis: q is converted in the same one, and the
// columns of O are put back when a partial is stored.
struct PxRaw {
    uint32_t v[4][4], sc[4];
};
// Loads into registers that hold something already ("+"): written so, the two
// branches that fetch (entries, window rows) share the registers, and no move
// after them waits for a load.
__device__ __forceinline__ void px_ld16(uint32_t (&v)[4], const void *at) {
    asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];" : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]) : "l"(at));
}
__device__ __forceinline__ void px_ld4(uint32_t &v, const void *at) { asm volatile("ld.global.nc.u32 %0, [%1];" : "+r"(v) : "l"(at)); }
// Units u0 and u0 + 1 of a run: `row` the lane's, the second unit ROWS rows and
// VALUES values further on.
template <int ROWS, int VALUES>
__device__ __forceinline__ void px_fetch_run(const PrefixParams &p, int64_t row, int d0, PxRaw &raw, int u0) {
    const uint8_t *at = p.kv.codes + row * (CSA2_D / 2) + d0 / 2;
    // the aligned word that holds the unit's two scales
    const uint8_t *sc = p.kv.scales + row * (CSA2_D / CSA2_BLOCK) + ((d0 / CSA2_BLOCK) & ~3);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        px_ld16(raw.v[u0 + u], at + u * (ROWS * (CSA2_D / 2) + VALUES / 2));
        px_ld4(raw.sc[u0 + u], sc + u * (ROWS * (CSA2_D / CSA2_BLOCK) + VALUES / CSA2_BLOCK));
    }
}
// Four matrices of 8 rows by 16 bytes; lane l gives the address of row l % 8 of
// matrix l / 8.
__device__ __forceinline__ void px_stm(uint32_t addr, const uint32_t (&h)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3])
                 : "memory");
}
// Matrices 4 j .. 4 j + 3 of a unit: a block of 64 positions is a 128-byte row,
// swizzled by its number, so matrices 4 to 7 lie 64 bytes across from 0 to 3
// (addr's own swizzle included) and 8 to 15 in the next block.
__device__ __forceinline__ uint32_t px_matrix(uint32_t addr, int j, uint32_t block) { return (j & 1 ? addr ^ 64u : addr) + (j >> 1) * block; }
// Words of FP4 codes and the unit's two scales -> f16 pairs -> matrices.
__device__ __forceinline__ void px_store_fp4(const uint32_t (&w)[4], uint32_t sc, uint32_t addr, uint32_t block) {
    const uint32_t s2 = e4m3x2_to_f16x2((uint16_t)sc);
    const uint32_t f[2] = {__byte_perm(s2, 0, 0x1010), __byte_perm(s2, 0, 0x3232)};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t h[4];
        e2m1x8_to_f16x8(w[j], h);
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = hmul2_u32(h[k], f[j >> 1]);
        px_stm(px_matrix(addr, j, block), h);
    }
}
// Pairs of a window row's unit: its first 16 bytes (raw) and its last (m).
__device__ __forceinline__ void px_pairs_e4m3(const uint32_t (&raw)[4], const uint4 &m, uint32_t (&h)[16]) {
    const uint32_t w[8] = {raw[0], raw[1], raw[2], raw[3], m.x, m.y, m.z, m.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        h[2 * j] = e4m3x2_to_f16x2((uint16_t)(w[j] & 0xFFFFu));
        h[2 * j + 1] = e4m3x2_to_f16x2((uint16_t)(w[j] >> 16));
    }
}
__device__ __forceinline__ void px_store_pairs(const uint32_t (&h)[16], uint32_t addr, uint32_t block) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t x[4] = {h[4 * j], h[4 * j + 1], h[4 * j + 2], h[4 * j + 3]};
        px_stm(px_matrix(addr, j, block), x);
    }
}

// Entries that row r of a strip sees of the strip's list; -1 where there is no
// such row.
__device__ __forceinline__ int32_t px_sees(const PrefixParams &p, const PrefixStrip &t, int r) {
    if (r >= t.q_rows) return -1;
    if (t.member0 < 0) return t.rows;
    const int32_t x = t.row0 + r, per = p.q_per_seq * p.h;
    const int32_t j = x / per, y = x - j * per;
    const int32_t s = p.members[t.member0 + j];
    if (s < 0 || s >= p.kv.batch) return -1;
    const int64_t u = (int64_t)s * p.q_per_seq + y / p.h;
    return u < p.nq ? min(px_limit(p, s, u), t.rows) : -1;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPxThreads, 1) k_prefix_attn(const __grid_constant__ CUtensorMap q_map, PrefixParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *q_s = base;                         // [8 blocks of 64 values][64 rows][128 B]
    uint8_t *p_s = q_s + kPxQBytes;              // [4 blocks of 64 cache rows][64 rows][128 B]
    uint8_t *ring = p_s + kPxPBytes;             // [kPxSlots][32 KiB]
    uint8_t *misc = ring + kPxSlots * kPxSlotBytes;
    // The first CTA's full, p_full and q_full are what the products wait for:
    // the warps of both CTAs arrive at them. The others are signalled in both.
    uint64_t *full = reinterpret_cast<uint64_t *>(misc);  // [kPxSlots]
    uint64_t *p_full = full + kPxSlots;
    uint64_t *q_full = p_full + 1;
    uint64_t *empty = q_full + 1;         // [kPxSlots]
    uint64_t *s_full = empty + kPxSlots;  // [2]
    uint64_t *pv_done = s_full + 2;
    uint64_t *info_full = pv_done + 1;         // [kPxInfos]
    uint64_t *info_empty = info_full + kPxInfos;  // [kPxInfos]
    uint64_t *q_copy = info_empty + kPxInfos;     // [2], the second unused
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(q_copy + 2);
    PxInfo *infos = reinterpret_cast<PxInfo *>(tmem_slot + 2);   // [kPxInfos]
    float *xch = reinterpret_cast<float *>(infos + kPxInfos);    // [2][128] maxima of even and odd tiles
    constexpr int kBars = 2 * kPxSlots + 5 + 2 * kPxInfos + 2;
    static_assert(8 * kBars + 8 + kPxInfos * sizeof(PxInfo) + 1024 <= kPxMisc && (8 * kBars + 8) % 16 == 0, "misc");

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank();
    pdl_trigger();
    if (warp == 0) {
        tmem_alloc2(tmem_slot, 512);
        tmem_relinquish2();
    }
    if (tid == 0) {
        for (int i = 0; i < kPxSlots; ++i) {
            mbar_init(&full[i], kPxLoadWarps / 2);  // one set of each CTA
            mbar_init(&empty[i], 1);
        }
        mbar_init(&s_full[0], 1);
        mbar_init(&s_full[1], 1);
        mbar_init(pv_done, 1);
        mbar_init(p_full, 2 * kPxSoftWarps);
        mbar_init(q_full, 2);
        mbar_init(q_copy, 1);
        for (int i = 0; i < kPxInfos; ++i) {
            mbar_init(&info_full[i], 1);
            mbar_init(&info_empty[i], kPxLoadWarps + kPxSoftWarps);
        }
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // both CTAs' barriers are initialised, both TMEMs allocated
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();

    const int32_t c = blockIdx.x >> 1;
    const int32_t pairs = px_pairs(p.pairs, p.total_tiles[1]);
    const int64_t x0 = c < pairs ? p.start_tile[c] : 0;
    const int n = c < pairs ? (int)(p.start_tile[c + 1] - x0) : 0;
    constexpr uint32_t kColS = 256;

    if (warp >= kPxMmaWarp) {
        regs_dec<40>();
        if (n > 0 && warp == kPxMmaWarp && rank == 0) {
            // The whole warp walks and waits, one elected lane issues: descriptors
            // stay in uniform registers that way (64 cycles an instruction or less;
            // from a branch of lane 0 alone an instruction took 65 and more to issue,
            // which bounded the kernel).
            // Waits of CTA scope although the second CTA's arrivals count too: this
            // warp loads none of what they announce, the tensor cores read it through
            // the async proxy, for which the writers fenced. (Acquiring at cluster
            // scope takes some 250 cycles more a wait.)
            constexpr uint32_t idesc_s = idesc_f16_f32(128, 256, 0, 0), idesc_o = idesc_f16_f32(128, 256, 0, 1);
            const uint64_t a_q = make_sdesc(smem_u32(q_s), 16, 1024, kSw128);
            const uint64_t a_p = make_sdesc(smem_u32(p_s), 16, 1024, kSw128);
            const uint64_t b_k = make_sdesc(smem_u32(ring), 16, 1024, kSw128);
            const uint64_t b_v = make_sdesc(smem_u32(ring), 8192, 1024, kSw128);
            PxWalk wk, wv;  // tiles of S and of P V
            wk.begin(p, c, x0);
            wv = wk;
            uint32_t chunk = 0, strips = 0;
            bool ok = true;
            auto scores = [&](int i) {
                if (i == 0 || wk.tile == 0) ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait(q_full, strips++ & 1u));
#pragma unroll 1
                for (int d = 0; d < 4 && ok; ++d, ++chunk) {
                    const uint32_t slot = chunk % kPxSlots;
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(&full[slot], (chunk / kPxSlots) & 1u));
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t a = a_q + (uint64_t)(d * 16384 >> 4), b = b_k + (uint64_t)(slot * kPxSlotBytes >> 4);
                    const uint32_t to = tmem + kColS + 128 * (i & 1);
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)  // two blocks of 64 values
                            mma_f16_pair(to, a + (uint64_t)(((k >> 2) * 8192 + (k & 3) * 32) >> 4),
                                         b + (uint64_t)(((k >> 2) * 16384 + (k & 3) * 32) >> 4), idesc_s, (d | k) ? 1u : 0u);
                        tc_commit_pair(&empty[slot]);
                        if (d == 3) tc_commit_pair(&s_full[i & 1]);
                    }
                    __syncwarp();
                }
            };
            scores(0);
            for (int i = 0; i < n && ok; ++i) {
                if (i + 1 < n) {
                    wk.next(p);
                    scores(i + 1);
                }
                ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait(p_full, (uint32_t)i & 1u));
                const uint32_t fresh = i == 0 || wv.tile == 0;
                const int nv = wv.value_chunks();
#pragma unroll 1
                for (int d = 0; d < nv && ok; ++d, ++chunk) {
                    const uint32_t slot = chunk % kPxSlots;
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(&full[slot], (chunk / kPxSlots) & 1u));
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t a = a_p + (uint64_t)(d * 8192 >> 4), b = b_v + (uint64_t)(slot * kPxSlotBytes >> 4);
                    const uint32_t add = fresh && d == 0 ? 0u : 1u;
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                mma_f16_pair(tmem + 128 * j, a + (uint64_t)(k * 32 >> 4), b + (uint64_t)((j * 16384 + k * 2048) >> 4), idesc_o,
                                             k > 0 ? 1u : add);
                        tc_commit_pair(&empty[slot]);
                        if (d == nv - 1) tc_commit_pair(pv_done);
                    }
                    __syncwarp();
                }
                if (i + 1 < n) wv.next(p);
            }
        } else if (n > 0 && warp == kPxMmaWarp + 1) {
            // ---- resolver: lane g has run g of each tile ----
            PxWalk w;
            w.begin(p, c, x0);
            bool ok = true;
            for (int i = 0; i < n && ok; ++i) {
                const int slot = i % kPxInfos;
                const int32_t j = w.tile * kPxTile + 16 * (lane & 15);
                PxLook x;
                px_look(p, w.t, w.tile, 16 * (lane & 15), x);
                int32_t base = j >= w.t.rows ? kPxNone : kPxMixed;
                if (j >= w.t.entries && j + 16 <= w.t.rows && (int64_t)(-2 - x.code) + 16 <= p.swa_seq_stride) base = kPxWindow + 2 + x.code;
                if (j + 16 <= w.t.entries && x.code + 16 <= p.kv.page_size) {
                    const int64_t row = (int64_t)x.page * p.kv.page_size + x.code;
                    if (x.page >= 0 && row + 16 <= p.kv.rows_cap) base = (int32_t)row;
                }
                uint32_t have = base >= 0 || base <= kPxWindow ? 0xFFFFu : 0u;
                uint32_t mixed = __ballot_sync(0xFFFFFFFFu, base == kPxMixed) & 0xFFFFu;
                while (mixed) {
                    const int g = __ffs(mixed) - 1;
                    mixed &= mixed - 1;
                    PxLook y;
                    px_look(p, w.t, w.tile, 16 * g + (lane & 15), y);
                    const uint32_t m = __ballot_sync(0xFFFFFFFFu, px_row(p, y) != kPxNone) & 0xFFFFu;
                    if ((lane & 15) == g) have = m;
                }
                if (i >= kPxInfos) ok = __all_sync(0xFFFFFFFFu, mbar_wait(&info_empty[slot], (uint32_t)(i / kPxInfos - 1) & 1u));
                if (!ok) break;
                PxInfo &f = infos[slot];
                if (lane < 16) {
                    f.base[lane] = base;
                    reinterpret_cast<uint16_t *>(f.valid)[lane] = (uint16_t)have;
                }
                if (lane == 0) {
                    f.tile = w.tile;
                    f.left = min(kPxTile, w.t.rows - w.tile * kPxTile);
                    f.seq = w.t.seq;
                    f.t_base = w.t.t_base;
                    f.entries = w.t.entries;
                    f.rows = w.t.rows;
                    f.w_begin = w.t.w_begin;
                    f.w_seq = w.t.w_seq;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&info_full[slot]);
                if (i + 1 < n) w.next(p);
            }
        } else if (n > 0 && warp == kPxMmaWarp + 2) {
            // ---- q of each strip, once S of the last tile before is done ----
            const uint32_t q_full_addr = cluster_smem_addr(q_full, 0);
            PxWalk w;
            w.begin(p, c, x0);
            bool ok = true;
            uint32_t copies = 0;
            for (int i = 0; i < n && ok; ++i) {
                if (i == 0 || w.tile == 0) {
                    if (w.t.q_rows > 64 * (int)rank) {
                        if (lane == 0) {
                            mbar_arrive_expect_tx(q_copy, kPxQBytes);
                            for (int b = 0; b < 8; ++b) tma_load_2d(q_s + b * 8192, &q_map, q_copy, 64 * b, w.t.q_at + 64 * (int)rank);
                        }
                        __syncwarp();
                        ok = __all_sync(0xFFFFFFFFu, mbar_wait(q_copy, copies & 1u));
                        ++copies;
                    }
                    if (ok && lane == 0) mbar_arrive_pair(q_full_addr);
                }
                // every phase of s_full is waited for, so that none is mistaken for another
                if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait(&s_full[i & 1], ((uint32_t)i >> 1) & 1u));
                if (i + 1 < n) w.next(p);
            }
        }
        __syncwarp();
    } else if (warp >= kPxSoftWarps) {
        regs_dec<72>();
        if (n > 0) {
        // ---- rows of the cache into the ring: four sets of four warps, a slot of
        // the ring each, so that a set never waits for a phase that another has
        // yet to begin. Chunk x of the call goes to slot x % 4. Lane l of a warp has
        //   keys: rows 8 u + l / 4 of the warp's 32, values 32 (l % 4) .. of the chunk's
        //     128;
        //   values: rows 8 (u / 2) + l / 4 of its 16, values 128 (u % 2) + 32 (l % 4) ..
        //     of the CTA's 256 ----
        const int set = (warp - kPxSoftWarps) >> 2, lw = (warp - kPxSoftWarps) & 3;
        const uint32_t full_addr = cluster_smem_addr(&full[set], 0);
        const int sub = lane >> 2;
        // row lane % 8 of matrix lane / 8, in the slot, swizzled
        const uint32_t stm_addr = smem_u32(ring) + set * kPxSlotBytes + (lane & 7) * 128 + (((lane >> 3) ^ (lane & 7)) << 4);
        PxRaw raw;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            raw.sc[u] = 0u;
#pragma unroll
            for (int j = 0; j < 4; ++j) raw.v[u][j] = 0u;
        }
        // The group whose chunk is in raw: entries or window rows in whole runs, or
        // rows that are resolved and loaded when the chunk is stored. What else the
        // later steps need of its tile they read again from its info.
        enum { kRunEntries, kRunWindow, kRows } kind = kRunEntries;
        bool keys = true, skip = false;
        int d = set;  // which of the group's chunks is the set's
        auto value0 = [&]() {
            return (keys ? 128 * d : 256 * (int)rank) + 32 * (lane & 3);
        };
        // The window ring of a tile; of a run of window rows, the lane's first unit.
        auto ring_of = [&](const PxInfo &f) { return p.swa + (int64_t)f.w_seq * p.swa_seq_stride * CSA2_D; };
        auto run_of = [&](const PxInfo &f) {
            const int32_t b0 = f.base[keys ? 8 * (int)rank + 2 * lw : 4 * d + lw];
            return ring_of(f) + (int64_t)(kPxWindow - b0 + sub) * CSA2_D + value0();
        };
        auto window_step = [&](int u) { return keys ? u * 8 * CSA2_D : (u >> 1) * 8 * CSA2_D + (u & 1) * 128; };
        // Fetches the set's chunk of tile i's keys or values, a group whose first
        // chunk is number `first`.
        auto fetch = [&](int i, bool of_keys, uint32_t first) {
            const PxInfo &f = infos[i % kPxInfos];
            keys = of_keys;
            d = (int)((set - first) & 3u);
            skip = !keys && 64 * d >= f.left;
            const int32_t b0 = f.base[keys ? 8 * (int)rank + 2 * lw : 4 * d + lw], b1 = keys ? f.base[8 * (int)rank + 2 * lw + 1] : b0;
            kind = b0 >= 0 && b1 >= 0 ? kRunEntries : b0 <= kPxWindow && (keys ? b1 == b0 - 16 : true) ? kRunWindow : kRows;
            const int d0 = value0();
            if (kind == kRunEntries) {
                if (keys) {
                    px_fetch_run<8, 0>(p, (int64_t)b0 + sub, d0, raw, 0);
                    px_fetch_run<8, 0>(p, (int64_t)b1 + sub, d0, raw, 2);
                } else {
                    px_fetch_run<0, 128>(p, (int64_t)b0 + sub, d0, raw, 0);
                    px_fetch_run<0, 128>(p, (int64_t)b0 + 8 + sub, d0, raw, 2);
                }
            } else if (kind == kRunWindow && !skip) {
                const uint8_t *at = run_of(f);
#pragma unroll
                for (int u = 0; u < 4; ++u) px_ld16(raw.v[u], at + window_step(u));
            }
        };
        bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(&info_full[0], 0));
        uint32_t chunk = 0, round = 0;  // first of the group; the slot's uses so far
        fetch(0, true, 0);
        // Groups in the order of the products: K(0), K(1), V(0), K(2), V(1), ...,
        // K(n - 1), V(n - 2), V(n - 1)
#pragma unroll 1
        for (int j = 0; j < 2 * n && ok; ++j) {
            const int tile = j == 0 ? 0 : j == 2 * n - 1 ? n - 1 : j & 1 ? (j + 1) / 2 : j / 2 - 1;
            const int chunks = keys ? 4 : (infos[tile % kPxInfos].left + 63) >> 6;
            if (!skip) {
                if (round > 0) ok = __all_sync(0xFFFFFFFFu, mbar_wait(&empty[set], (round - 1) & 1u));
                if (!ok) break;
                ++round;
                // blocks of 64 positions: keys [128 rows][128 B], values [64 rows][128 B]
                const uint32_t block = keys ? 16384u : 8192u;
                const uint32_t at0 = stm_addr + (uint32_t)lw * (keys ? 4096u : 2048u);
                auto unit = [&](int u) { return at0 + (keys ? u * 1024u : (u >> 1) * 1024u + (u & 1) * 16384u); };
                if (kind == kRunEntries) {
#pragma unroll
                    for (int u = 0; u < 4; ++u) px_store_fp4(raw.v[u], raw.sc[u] >> (16 * (lane & 1)), unit(u), block);
                } else if (kind == kRunWindow) {
                    // the second halves of the units, of sectors that the first ones brought
                    const uint8_t *at = run_of(infos[tile % kPxInfos]) + 16;
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        uint32_t h[16];
                        px_pairs_e4m3(raw.v[u], __ldg(reinterpret_cast<const uint4 *>(at + window_step(u))), h);
                        px_store_pairs(h, unit(u), block);
                    }
                } else {  // few chunks: resolved (a row a lane) and loaded only here, which spares registers
                    const PxInfo &f = infos[tile % kPxInfos];
                    PxLook look;
                    px_look(p, f, f.tile, keys ? 128 * (int)rank + 32 * lw + lane : 64 * d + 16 * lw + (lane & 15), look);
                    const int32_t rows = px_row(p, look);
#pragma unroll 1
                    for (int u = 0; u < 4; ++u) {
                        const int32_t src = __shfl_sync(0xFFFFFFFFu, rows, (keys ? 8 * u : 8 * (u >> 1)) + sub);
                        const int d0 = value0() + (keys ? 0 : 128 * (u & 1));
                        uint32_t h[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) h[k] = 0u;
                        if (src >= 0) {
                            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p.kv.codes + (int64_t)src * (CSA2_D / 2) + d0 / 2));
                            const uint32_t s2 = e4m3x2_to_f16x2(
                                __ldg(reinterpret_cast<const uint16_t *>(p.kv.scales + (int64_t)src * (CSA2_D / CSA2_BLOCK) + d0 / CSA2_BLOCK)));
                            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                uint32_t x[4];
                                e2m1x8_to_f16x8(w[j], x);
#pragma unroll
                                for (int k = 0; k < 4; ++k) h[4 * j + k] = hmul2_u32(x[k], __byte_perm(s2, 0, j < 2 ? 0x1010 : 0x3232));
                            }
                        } else if (src != kPxNone) {
                            const uint8_t *at = ring_of(f) + (int64_t)(-2 - src) * CSA2_D + d0;
                            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(at));
                            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                            px_pairs_e4m3(w, __ldg(reinterpret_cast<const uint4 *>(at + 16)), h);
                        }
                        __syncwarp();
                        px_store_pairs(h, unit(u), block);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_pair(full_addr);
            }
            chunk += chunks;
            if (!keys) {  // the tile's last use of its info
                __syncwarp();
                if (lane == 0) mbar_arrive(&info_empty[tile % kPxInfos]);
            }
            if (j + 1 < 2 * n) {
                const int nj = j + 1;
                const bool next_keys = (nj & 1) && nj != 2 * n - 1;
                const int nt = nj == 2 * n - 1 ? n - 1 : nj & 1 ? (nj + 1) / 2 : nj / 2 - 1;
                if (next_keys) ok = __all_sync(0xFFFFFFFFu, mbar_wait(&info_full[nt % kPxInfos], (uint32_t)(nt / kPxInfos) & 1u));
                if (!ok) break;
                fetch(nt, next_keys, chunk);
            }
        }
        }
    } else {
        regs_inc<152>();
        if (n > 0) {
        // ---- softmax: this thread has row 64 * rank + (tid & 63) of a strip and half of its scores ----
        const int r = tid & 63, half = tid >> 6;
        const uint32_t lane_addr = tmem + ((uint32_t)(warp * 32) << 16);
        const uint32_t p_full_addr = cluster_smem_addr(p_full, 0);
        const int pair_bar = 1 + (warp & 1);  // warps w and w + 2 have the same rows
        PxWalk w;
        w.begin(p, c, x0);
        bool ok = true;
        int32_t sees = px_sees(p, w.t, 64 * rank + r), next_sees = -1;
        float m_run = -INFINITY, l_run = 0.0f;
        // after a wait that gave up the loop goes on without waiting: the other
        // warps count on this one at their barriers
        for (int i = 0; i < n; ++i) {
            const bool last = i == n - 1 || w.last();
            const int lim = min(max(sees - w.tile * kPxTile - 128 * half, 0), 128);
            // where the strip's partial goes (used when last)
            const bool pre = w.t.member0 >= 0;
            const int64_t part = pre ? ((int64_t)c + w.s) * kPxRows + 64 * rank + r : ((int64_t)c + (w.s - w.n_pre)) * p.h + 64 * rank + r;
            // what the resolver tells of the tile is read below: S being done does not
            // order its plain stores before that (told long before S: no time is lost)
            if (ok) ok = mbar_wait(&info_full[i % kPxInfos], (uint32_t)(i / kPxInfos) & 1u);
            if (ok) ok = mbar_wait(&s_full[i & 1], ((uint32_t)i >> 1) & 1u);
            tc_fence_after();
            if (i + 1 < n) {
                w.next(p);
                if (last) next_sees = px_sees(p, w.t, 64 * rank + r);
            }
            const uint32_t ts = lane_addr + kColS + 128 * (i & 1);
            // scores of this thread that do not count become -inf, in TMEM and by a
            // loop of its own, so that the common path has no masks
            const uint4 vw = *reinterpret_cast<const uint4 *>(infos[i % kPxInfos].valid + half * 4);
            __syncwarp();
            if (lane == 0) mbar_arrive(&info_empty[i % kPxInfos]);
            // (rows that are none need no masks: what becomes of them reaches no other row)
            if (__any_sync(0xFFFFFFFFu, sees >= 0 && (lim < 128 || (vw.x & vw.y & vw.z & vw.w) != 0xFFFFFFFFu))) {
#pragma unroll 1
                for (int k = 0; k < 4; ++k) {
                    const int m = lim - 32 * k;
                    const uint32_t word = k == 0 ? vw.x : k == 1 ? vw.y : k == 2 ? vw.z : vw.w;
                    const uint32_t bits = word & (m >= 32 ? 0xFFFFFFFFu : m <= 0 ? 0u : (1u << m) - 1u);
                    uint32_t v[32];
                    tmem_ld32(ts + 32 * k, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = bits >> j & 1u ? v[j] : 0xFF800000u;
                    tmem_st32(ts + 32 * k, v);
                }
                tmem_wait_st();
            }
            float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
                uint32_t v[32], y[32];
                tmem_ld32(ts + 32 * k, v);
                tmem_ld32(ts + 32 * k + 32, y);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; ++j) t4[j & 3] = fmaxf(t4[j & 3], fmaxf(__uint_as_float(v[j]), __uint_as_float(y[j])));
            }
            float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) * p.scale_log2;
            // the row's other half
            xch[(i & 1) * 128 + tid] = top;
            named_bar_sync(pair_bar, 64);
            top = fmaxf(top, xch[(i & 1) * 128 + (tid ^ 64)]);
            float alpha = 1.0f;
            const bool raise = top > m_run + kPxRescale || (m_run == -INFINITY && top > -INFINITY);
            if (raise) {
                if (m_run != -INFINITY) alpha = ex2(m_run - top);
                m_run = top;
                l_run *= alpha;
            }
            const float at = m_run == -INFINITY ? 0.0f : m_run - kPxBias;
            float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            uint32_t pk[32];
            auto exps = [&](int k0) {  // scores 32 k0 .. + 63
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    uint32_t v[32];
                    tmem_ld32(ts + 32 * (k0 + k), v);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float a = ex2(fmaf(__uint_as_float(v[2 * j]), p.scale_log2, -at));
                        const float b = ex2(fmaf(__uint_as_float(v[2 * j + 1]), p.scale_log2, -at));
                        sum[j & 3] += a + b;
                        // f16: 2^-11 relative, 2^-25 absolute (see kPxBias)
                        const __half2 hh = __floats2half2_rn(a, b);
                        pk[16 * k + j] = *reinterpret_cast<const uint32_t *>(&hh);
                    }
                }
            };
            auto put_p = [&](int blk) {
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    *reinterpret_cast<uint4 *>(p_s + (2 * half + blk) * 8192 + r * 128 + ((x ^ (r & 7)) << 4)) =
                        make_uint4(pk[4 * x], pk[4 * x + 1], pk[4 * x + 2], pk[4 * x + 3]);
            };
            // half of P in registers while the products of the tile before read the last one
            exps(0);
            if (i > 0 && ok) ok = mbar_wait(pv_done, (uint32_t)(i - 1) & 1u);
            tc_fence_after();
            put_p(0);
            exps(2);
            put_p(1);
            l_run += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            if (__any_sync(0xFFFFFFFFu, alpha != 1.0f)) {
#pragma unroll 1
                for (int k = 0; k < 256; k += 32) {
                    uint32_t v[32];
                    tmem_ld32(lane_addr + k, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * alpha);
                    tmem_st32(lane_addr + k, v);
                }
                tmem_wait_st();
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_pair(p_full_addr);
            if (last) {
                // the strip's partial of this run
                xch[(~i & 1) * 128 + tid] = l_run;
                named_bar_sync(pair_bar, 64);
                const float l = l_run + xch[(~i & 1) * 128 + (tid ^ 64)];
                named_bar_sync(pair_bar, 64);  // the next tile's maxima go there
                const float inv = l > 0.0f ? 1.0f / l : 0.0f;
                if (ok) ok = mbar_wait(pv_done, (uint32_t)i & 1u);
                tc_fence_after();
                // O / l through the P buffer (free now), 64 positions at a time (half of a
                // 128: matrices m0 .. m0 + 7): a thread has 256 bytes of its row there, in
                // 16-byte units turned by its lane; unit 4 q + t is values 32 q + 2 m0 + 4 t
                // .. + 3, and half a warp stores a row's units to their places
                const bool mine = ok && sees >= 0;
                const uint32_t whose = __ballot_sync(0xFFFFFFFFu, mine);
                uint8_t *stage = p_s + warp * 8192;
                float *dst = (pre ? p.pre_o : p.own_o) + (part - lane) * CSA2_D + 256 * half;
#pragma unroll 1
                for (int k = 0; k < 256; k += 64) {
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        uint32_t v[32];
                        tmem_ld32(lane_addr + k + 32 * y, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                        {
                            // positions 32 y + 8 m + 2 q + e: this half's matrices 4 y + m
                            const int q = j & 3, t = j >> 2;  // matrices 2 t, 2 t + 1 of the four
                            *reinterpret_cast<float4 *>(stage + lane * 256 + (((4 * q + 2 * y + t) ^ (lane & 15)) << 4)) =
                                make_float4(__uint_as_float(v[16 * t + 2 * q]) * inv, __uint_as_float(v[16 * t + 2 * q + 1]) * inv,
                                            __uint_as_float(v[16 * t + 8 + 2 * q]) * inv, __uint_as_float(v[16 * t + 9 + 2 * q]) * inv);
                        }
                    }
                    __syncwarp();
#pragma unroll
                    for (int j0 = 0; j0 < 16; j0 += 8) {
                        float4 o[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const int row = 2 * (j0 + j) + (lane >> 4);
                            o[j] = *reinterpret_cast<const float4 *>(stage + row * 256 + (((lane ^ row) & 15) << 4));
                        }
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const int row = 2 * (j0 + j) + (lane >> 4);
                            if (whose >> row & 1u)
                                __stcg(reinterpret_cast<float4 *>(dst + (int64_t)row * CSA2_D + (k & 128) + 32 * ((lane >> 2) & 3) + (k & 64) / 4) + (lane & 3), o[j]);
                        }
                    }
                    __syncwarp();
                }
                if (mine && half == 0)
                    (pre ? p.pre_lse : p.own_lse)[part] = l > 0.0f ? (m_run - kPxBias + log2f(l)) * 0.69314718055994531f : -INFINITY;
                tc_fence_before();
                m_run = -INFINITY;
                l_run = 0.0f;
                sees = next_sees;
                named_bar_sync(3, kPxSoftWarps * 32);  // P may be written again
            }
        }
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // no CTA of the pair leaves while the other's products or arrivals reach it
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc2(*reinterpret_cast<volatile uint32_t *>(tmem_slot), 512);  // read again: no register across the roles
    }
}

// ---------------------------------------------------------------------------
// merge: one block per (member, query, head): o = sum_s w_s o_s / sum_s w_s,
// w_s = exp(lse_s - max), over the partials of its prefix strip and its own.
// ---------------------------------------------------------------------------
constexpr int kPxMergeThreads = 128;
constexpr int kPxMergeParts = 512;  // at most two strips over all pairs

__global__ void __launch_bounds__(kPxMergeThreads) k_prefix_merge(PrefixParams p) {
    __shared__ float wgt[kPxMergeParts];
    __shared__ float red[2][4];
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x;
    const int32_t i = blockIdx.x, head = blockIdx.y;
    const PrefixItem item = p.items[i];
    const int64_t cost = p.total_tiles[1];
    const int32_t pairs = px_pairs(p.pairs, cost);
    if (item.u < 0) return;
    const int64_t u = item.u;
    int32_t na = 0, nb = 0;
    int64_t a0 = 0, b0 = 0;  // first rows of the partials
    if (item.pre_tiles > 0) {
        const int32_t x = item.x0 + head, s = x / kPxRows;
        const int64_t c0 = item.pre_cost0 + (int64_t)s * (item.pre_tiles + kPxStripCost);
        const int32_t c = px_owner(cost, pairs, c0, 0);
        na = px_owner(cost, pairs, c0, item.pre_tiles - 1) - c + 1;
        a0 = ((int64_t)c + item.pre_strip + s) * kPxRows + x % kPxRows;
    }
    if (item.own_tiles > 0) {
        const int32_t c = px_owner(cost, pairs, item.own_cost0, 0);
        nb = px_owner(cost, pairs, item.own_cost0, item.own_tiles - 1) - c + 1;
        b0 = ((int64_t)c + i) * p.h + head;
    }
    const int32_t np = na + nb;
    if (np > kPxMergeParts) {
        if (tid == 0) set_error(CSA2_DEVERR_SELECT);
        return;
    }
    float top = -INFINITY;
    for (int s = tid; s < np; s += kPxMergeThreads) {
        const float v = s < na ? p.pre_lse[a0 + (int64_t)s * kPxRows] : p.own_lse[b0 + (int64_t)(s - na) * p.h];
        wgt[s] = v;
        top = fmaxf(top, v);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    if ((tid & 31) == 0) red[0][tid >> 5] = top;
    __syncthreads();
    top = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
    float sum = 0.0f;
    for (int s = tid; s < np; s += kPxMergeThreads) {
        const float v = top == -INFINITY ? 0.0f : expf(wgt[s] - top);
        wgt[s] = v;
        sum += v;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if ((tid & 31) == 0) red[1][tid >> 5] = sum;
    __syncthreads();
    sum = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kBatch = 8;
    for (int s1 = 0; s1 < np; s1 += kBatch) {
        float4 v[kBatch];
#pragma unroll
        for (int s = 0; s < kBatch; ++s) {
            const int x = s1 + s;
            if (x < np)
                v[s] = *(reinterpret_cast<const float4 *>(x < na ? p.pre_o + (a0 + (int64_t)x * kPxRows) * CSA2_D
                                                                 : p.own_o + (b0 + (int64_t)(x - na) * p.h) * CSA2_D) + tid);
        }
#pragma unroll
        for (int s = 0; s < kBatch; ++s)
            if (s1 + s < np) {
                const float w = wgt[s1 + s];
                acc.x = fmaf(w, v[s].x, acc.x);
                acc.y = fmaf(w, v[s].y, acc.y);
                acc.z = fmaf(w, v[s].z, acc.z);
                acc.w = fmaf(w, v[s].w, acc.w);
            }
    }
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    const int64_t row = u * p.h + head;
    const uint32_t lo = (uint32_t)f32_to_bf16_bits(acc.x * inv) | ((uint32_t)f32_to_bf16_bits(acc.y * inv) << 16);
    const uint32_t hi = (uint32_t)f32_to_bf16_bits(acc.z * inv) | ((uint32_t)f32_to_bf16_bits(acc.w * inv) << 16);
    *(reinterpret_cast<uint2 *>(p.o + row * CSA2_D) + tid) = make_uint2(lo, hi);
    if (tid == 0 && p.lse) p.lse[row] = sum > 0.0f ? top + logf(sum) : -INFINITY;
}

}  // namespace csa2
