// pages.cuh -- the page operators of the paged global KV cache: copying,
// forking, resizing (growing, rolling back, freeing) and compacting.
//
// DeepSeek V4.1-Flash Cuts KV Cache by 437x (ainewsfeed.tech), paragraph
// "CSA2 tackles storage": one global KV shared by all layers, so a sequence
// is one row of the page table and its pages hold codes, scales and indexer
// keys of every layer. Several sequences may hold the same physical page;
// refs[p] counts them and 0 means free. The lowest free pages are taken
// first, so the state needs no free list and every result is a function of
// the arguments alone (no atomic's order shows).
//
// Each operator is a plan and an apply launch:
//   * plan: one cluster of kPlanCtas CTAs reads refs once (every CTA a run of
//     pages), the first CTA walks the entries of the call (how many new pages
//     each needs, an exclusive sum in the order of the entries), and the free
//     pages of rank 0, 1, ... are written to the workspace. A cluster rather
//     than a grid, because the ranks need the counts of all runs before and
//     distributed shared memory gives them within the launch.
//   * apply: the whole grid writes table rows and counts and moves the bytes,
//     which is what bounds large calls (2 x rows x (288 + di) bytes). The plan of
//     a small fork or resize does that itself, after a cluster barrier, and
//     saves a launch (four forks of a 2000-entry sequence: 15.1 -> 11.7 us).
#pragma once

#include "common.cuh"

namespace csa2 {

constexpr int kPlanCtas = 8;  // the portable cluster size
constexpr int kPlanThreads = 1024;
constexpr int kApplyThreads = 256;
constexpr int kCopyUnitRows = 8;  // rows a warp moves at a time: 2 KiB of codes, 256 B of scales, 8 di of keys

// One entry of a fork or resize call as planned (the workspace's first array).
// A partial last page that has to become the sequence's own is a copy of the
// first part_rows rows of `from` (a fork's last page, or a shared page that a
// resize cut): the first page taken.
struct __align__(16) PageEntry {
    int32_t length;     // entries of the sequence afterwards; -1: refused
    int32_t had;        // entries before
    int32_t need;       // pages to take
    int32_t base;       // rank of the first one among the free pages
    int32_t from;       // page to copy in part
    int32_t part_rows;  // its rows; 0: no copy
    int32_t pad[2];
};

struct PagesParams {
    csa2_kv_desc kv;
    int32_t *table, *seq_len, *refs;
    int32_t num_pages, n;
    int32_t group_log2;  // log2 of the plan's threads for an entry, where it applies what it planned; -1: the apply launch does
    const int32_t *from;    // fork: parents
    const int32_t *to;      // fork: children; resize: sequences
    const int32_t *length;  // fork: entries to share (nullable); resize: new lengths
    int32_t *copy_src, *copy_dst;  // fork, resize: nullable [n]; compact: moves [num_pages / 2]
    int32_t *n_live;               // compact (nullable)
    // workspace
    int32_t *head;     // [4]: free pages, pages needed; compact: live pages, moves
    int32_t *claim;    // [batch]: the first entry that names a sequence
    PageEntry *entry;  // [n]
    int32_t *fresh;    // [num_pages]: free pages by rank; compact: a moved page's new number
};

__device__ __forceinline__ int32_t pages_of(int32_t len, int32_t ps) { return len / ps + (len % ps != 0); }

// Exclusive sum over the block (kPlanThreads threads) and its total. A warp's sum is
// cut at `cap`: summands and cap of up to 2^26 (pages of a cache, and one more)
// keep every sum below 2^32, a result up to cap is exact, and one above stays above.
__device__ __forceinline__ uint32_t block_exclusive(uint32_t v, uint32_t *warp_sums, uint32_t &total, uint32_t cap = 0xFFFFFFFFu) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, s, o);
        if (lane >= o) s += u;
    }
    if (lane == 31) warp_sums[warp] = min(s, cap);
    __syncthreads();
    if (warp == 0) {
        uint32_t w = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, w, o);
            if (lane >= o) w += u;
        }
        warp_sums[lane] = w;
    }
    __syncthreads();
    const uint32_t before = (warp ? warp_sums[warp - 1] : 0) + s - v;
    total = warp_sums[31];
    __syncthreads();
    return before;
}
static_assert(kPlanThreads == 1024, "block_exclusive sums 32 warps");

// What every CTA of the plan tells the others.
struct PlanShared {
    uint32_t warp_sums[32];
    int32_t count[2];  // pages of this CTA's run that count (two kinds)
    int32_t total_need;
};

// A thread's four pages of the run [lo, hi) in round k (page p0 + 0..3).
__device__ __forceinline__ int32_t plan_page(int32_t lo, int32_t k) {
    return lo + (k * kPlanThreads + (int32_t)threadIdx.x) * 4;
}
__device__ __forceinline__ int4 plan_refs(const int32_t *refs, int32_t p, int32_t hi) {
    // runs start at multiples of four, so one load takes four counts where refs
    // is 16-byte aligned; a tail is read page by page (-1: no page)
    if (p + 4 <= hi && (reinterpret_cast<uintptr_t>(refs) & 15) == 0) return *reinterpret_cast<const int4 *>(refs + p);
    return make_int4(p < hi ? refs[p] : -1, p + 1 < hi ? refs[p + 1] : -1, p + 2 < hi ? refs[p + 2] : -1, p + 3 < hi ? refs[p + 3] : -1);
}

// The two halves of cluster_sync_all().
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

// Sum of a count over the cluster's CTAs before this one, and over all.
__device__ __forceinline__ void cluster_sums(PlanShared &sh, int which, uint32_t rank, int32_t &before, int32_t &all) {
    before = all = 0;
    for (uint32_t c = 0; c < kPlanCtas; ++c) {
        const int32_t v = cluster_peer(&sh, c)->count[which];
        all += v;
        if (c < rank) before += v;
    }
}

// ---------------------------------------------------------------------------
// moving rows
// ---------------------------------------------------------------------------
// A warp copies rows [r0, r0 + kCopyUnitRows) of page `from` to page `to`,
// those below `rows`. All loads are issued before the first store.
__device__ __forceinline__ void copy_unit(const csa2_kv_desc &kv, int64_t from, int64_t to, int32_t r0, int32_t rows) {
    const int lane = threadIdx.x & 31;
    const int64_t a = from * kv.page_size + r0, b = to * kv.page_size + r0;
    const int32_t m = rows - r0;  // rows of the unit that move, if below kCopyUnitRows
    constexpr int kCodePieces = CSA2_D / 2 / 16;              // 16-byte pieces of a row: 16 of codes,
    constexpr int kScalePieces = CSA2_D / CSA2_BLOCK / 16;    // 2 of scales, di / 16 of keys
    constexpr int kC = kCopyUnitRows * kCodePieces / 32;
    const uint4 *cs = reinterpret_cast<const uint4 *>(kv.codes) + a * kCodePieces;
    uint4 *cd = reinterpret_cast<uint4 *>(kv.codes) + b * kCodePieces;
    const uint4 *ss = reinterpret_cast<const uint4 *>(kv.scales) + a * kScalePieces;
    uint4 *sd = reinterpret_cast<uint4 *>(kv.scales) + b * kScalePieces;
    const int kp = kv.kidx ? kv.di / 16 : 0;  // 4 or 8
    const uint4 *ks = reinterpret_cast<const uint4 *>(kv.kidx) + a * kp;
    uint4 *kd = reinterpret_cast<uint4 *>(kv.kidx) + b * kp;
    uint4 c[kC], s, k[2];
#pragma unroll
    for (int j = 0; j < kC; ++j) {
        const int x = lane + 32 * j;
        if (x / kCodePieces < m) c[j] = cs[x];
    }
    if (lane < kCopyUnitRows * kScalePieces && lane / kScalePieces < m) s = ss[lane];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int x = lane + 32 * j;
        if (x < kCopyUnitRows * kp && x < m * kp) k[j] = ks[x];
    }
#pragma unroll
    for (int j = 0; j < kC; ++j) {
        const int x = lane + 32 * j;
        if (x / kCodePieces < m) cd[x] = c[j];
    }
    if (lane < kCopyUnitRows * kScalePieces && lane / kScalePieces < m) sd[lane] = s;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int x = lane + 32 * j;
        if (x < kCopyUnitRows * kp && x < m * kp) kd[x] = k[j];
    }
}

// Pages src[i] -> dst[i] of a list, whole: the grid's warps stride over the
// units of all pages. n is p.n, or head[1] (the moves of a compaction).
__device__ __forceinline__ void copy_pages(const csa2_kv_desc &kv, const int32_t *src, const int32_t *dst, int64_t n,
                                           int32_t num_pages) {
    const int32_t per = kv.page_size / kCopyUnitRows;
    const int64_t W = (int64_t)gridDim.x * (kApplyThreads / 32);
    for (int64_t u = (int64_t)blockIdx.x * (kApplyThreads / 32) + (threadIdx.x >> 5); u < n * per; u += W) {
        const int64_t i = u / per;
        const int32_t r0 = (int32_t)(u - i * per) * kCopyUnitRows;
        const int32_t a = __ldcg(src + i), b = __ldcg(dst + i);
        if (a == -1 || b == -1 || a == b) continue;  // an empty slot
        if (a < 0 || b < 0 || a >= num_pages || b >= num_pages) {
            if (r0 == 0 && (threadIdx.x & 31) == 0) set_error(CSA2_DEVERR_BAD_ROW);
            continue;
        }
        copy_unit(kv, a, b, r0, kv.page_size);
    }
}

__global__ void __launch_bounds__(kApplyThreads) k_pages_copy(PagesParams p) {
    pdl_trigger();
    pdl_wait();
    copy_pages(p.kv, p.copy_src, p.copy_dst, p.n, p.num_pages);
}

// ---------------------------------------------------------------------------
// fork and resize: what is planned is done. Entries i0, i0 + istep, ...; thread t0
// of the step threads of an entry takes its share of the table row (a thread a
// column) and of the page copy (a warp a unit).
// ---------------------------------------------------------------------------
template <bool FORK>
__device__ __forceinline__ void pages_apply(const PagesParams &p, int32_t t0, int32_t step, int32_t i0, int32_t istep) {
    const int32_t ps = p.kv.page_size, width = p.kv.max_pages;
    const int32_t avail = __ldcg(p.head);
    const bool first = t0 == 0;
    for (int32_t i = i0; i < p.n; i += istep) {
        const PageEntry e = p.entry[i];
        const bool ok = e.length >= 0 && (e.need == 0 || (int64_t)e.base + e.need <= avail);
        if (!ok) {
            if (first) {
                set_error(CSA2_DEVERR_PAGES);
                if (p.copy_src) p.copy_src[i] = p.copy_dst[i] = -1;
            }
            continue;
        }
        const int32_t s = p.to[i];
        int32_t *row = p.table + (int64_t)s * width;
        const int32_t part = e.part_rows != 0;
        const int32_t into = part ? p.fresh[e.base] : -1;
        if (FORK) {
            const int32_t *src = p.table + (int64_t)p.from[i] * width;
            const uint32_t whole = (uint32_t)(e.length / ps);
            // unsigned: the last step may pass 2^31 in the widest rows
            for (uint32_t c = t0; c < (uint32_t)width; c += step) {
                int32_t page = -1;
                if (c < whole) {
                    page = src[c];
                    if (page < 0 || page >= p.num_pages) {
                        set_error(CSA2_DEVERR_BAD_ROW);
                        page = -1;
                    } else {
                        atomicAdd(p.refs + page, 1);
                    }
                } else if (c == whole && part) {
                    page = into;
                }
                row[c] = page;
            }
        } else {
            const int32_t had = pages_of(e.had, ps), has = pages_of(e.length, ps);
            for (int32_t c = min(had, has) + t0; c < max(had, has); c += step) {
                if (c >= has) {
                    const int32_t page = row[c];
                    if (page < 0 || page >= p.num_pages) set_error(CSA2_DEVERR_BAD_ROW);
                    else if (atomicSub(p.refs + page, 1) <= 0) set_error(CSA2_DEVERR_PAGES);
                    row[c] = -1;
                } else {
                    const int32_t page = p.fresh[e.base + part + (c - had)];
                    p.refs[page] = 1;
                    row[c] = page;
                }
            }
            // the cut page lies in front of the columns above
            if (part && t0 == 0) {
                atomicSub(p.refs + e.from, 1);
                row[min(e.length, e.had) / ps] = into;
            }
        }
        if (part) {
            const int64_t rows = (int64_t)(step / 32) * kCopyUnitRows;
            for (int64_t r = (t0 >> 5) * (int64_t)kCopyUnitRows; r < e.part_rows; r += rows)
                copy_unit(p.kv, e.from, into, (int32_t)r, e.part_rows);
        }
        if (first) {
            if (part) p.refs[into] = 1;
            p.seq_len[s] = e.length;
            if (p.copy_src) {
                p.copy_src[i] = part ? e.from : -1;
                p.copy_dst[i] = into;
            }
        }
    }
}

template <bool FORK>
__global__ void __launch_bounds__(kApplyThreads) k_pages_apply(PagesParams p) {
    pdl_trigger();
    pdl_wait();
    pages_apply<FORK>(p, blockIdx.x * kApplyThreads + threadIdx.x, gridDim.x * kApplyThreads, blockIdx.y, gridDim.y);
}

// ---------------------------------------------------------------------------
// fork and resize: the plan
// ---------------------------------------------------------------------------
constexpr PageEntry kRefused{-1, 0, 0, 0, -1, 0, {0, 0}};

template <bool FORK>
__device__ __forceinline__ PageEntry plan_entry(const PagesParams &p, int32_t i) {
    PageEntry e = kRefused;
    const int32_t ps = p.kv.page_size, batch = p.kv.batch;
    const int32_t s = p.to[i];
    if (s < 0 || s >= batch || __ldcg(p.claim + s) != i) return e;  // out of the batch, or named before
    const int64_t room = (int64_t)p.kv.max_pages * ps;
    const int32_t had = p.seq_len[s];
    int32_t len, cut, from_seq;  // the entries kept, and whose last page holds them
    if (FORK) {
        from_seq = p.from[i];
        if (from_seq < 0 || from_seq >= batch || from_seq == s || had != 0) return e;  // a child has to be empty
        len = p.seq_len[from_seq];
        if (p.length) len = min(len, p.length[i]);
        cut = len;
    } else {
        from_seq = s;
        len = p.length[i];
        if (had < 0 || had > room) return e;
        cut = min(len, had);
    }
    if (len < 0 || len > room) return e;
    if (cut % ps != 0) {
        e.from = p.table[(int64_t)from_seq * p.kv.max_pages + cut / ps];
        if (e.from < 0 || e.from >= p.num_pages) return e;
        if (FORK || p.refs[e.from] > 1) e.part_rows = cut % ps;
    }
    e.length = len;
    e.had = had;
    e.need = (e.part_rows != 0) + (FORK ? 0 : max(0, pages_of(len, ps) - pages_of(had, ps)));
    return e;
}

template <bool FORK>
__global__ void __launch_bounds__(kPlanThreads) k_pages_plan(PagesParams p) {
    __shared__ PlanShared sh;
    const uint32_t rank = cluster_rank();
    pdl_trigger();
    pdl_wait();
    if (rank == 0) {  // the entries, while the other CTAs count
        for (int32_t b = threadIdx.x; b < p.kv.batch; b += kPlanThreads) p.claim[b] = INT32_MAX;
        __syncthreads();
        for (int32_t i = threadIdx.x; i < p.n; i += kPlanThreads) {
            const int32_t s = p.to[i];
            if (s >= 0 && s < p.kv.batch) atomicMin(p.claim + s, i);
        }
        __syncthreads();
        int64_t sum = 0;
        for (int32_t i0 = 0; i0 < p.n; i0 += kPlanThreads) {
            const int32_t i = i0 + threadIdx.x;
            PageEntry e = kRefused;
            if (i < p.n) e = plan_entry<FORK>(p, i);
            uint32_t t;
            const uint32_t cap = (uint32_t)p.num_pages + 1;  // a need or a rank that no cache serves
            e.need = (int32_t)min((uint32_t)e.need, cap);
            const uint32_t before = block_exclusive((uint32_t)e.need, sh.warp_sums, t, cap);
            e.base = (int32_t)min(sum + before, (int64_t)cap);
            if (i < p.n) p.entry[i] = e;
            sum += t;
        }
        if (threadIdx.x == 0) sh.total_need = (int32_t)min(sum, (int64_t)p.num_pages);
    }
    const int32_t run = ((p.num_pages + kPlanCtas - 1) / kPlanCtas + 3) & ~3;
    const int32_t lo = min((int64_t)p.num_pages, (int64_t)rank * run), hi = min((int64_t)p.num_pages, (int64_t)lo + run);
    const int32_t rounds = (hi - lo + 4 * kPlanThreads - 1) / (4 * kPlanThreads);
    int32_t mine = 0;
    for (int32_t k = 0; k < rounds; ++k) {
        const int4 r = plan_refs(p.refs, plan_page(lo, k), hi);
        mine += (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0);
    }
    uint32_t total;
    block_exclusive(mine, sh.warp_sums, total);
    if (threadIdx.x == 0) sh.count[0] = (int32_t)total;
    cluster_sync_all();
    int32_t before, all;
    cluster_sums(sh, 0, rank, before, all);
    const int32_t need = min(cluster_peer(&sh, 0)->total_need, all);
    cluster_arrive();  // done with the other CTAs' shared memory
    if (rank == 0 && threadIdx.x == 0) {
        p.head[0] = all;
        p.head[1] = need;
    }
    for (int32_t k = 0; k < rounds && before < need; ++k) {
        const int32_t page = plan_page(lo, k);
        const int4 r = plan_refs(p.refs, page, hi);
        const int32_t f[4] = {r.x == 0, r.y == 0, r.z == 0, r.w == 0};
        uint32_t t;
        int32_t at = before + block_exclusive(f[0] + f[1] + f[2] + f[3], sh.warp_sums, t);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (f[j]) {
                if (at < need) p.fresh[at] = page + j;
                ++at;
            }
        before += t;
    }
    cluster_wait();  // no CTA leaves while another reads its shared memory
    if (p.group_log2 >= 0) {
        cluster_sync_all();  // the plan is in place
        const int32_t t = rank * kPlanThreads + threadIdx.x, group = 1 << p.group_log2;
        pages_apply<FORK>(p, t & (group - 1), group, t >> p.group_log2, (kPlanCtas * kPlanThreads) >> p.group_log2);
    }
}

// ---------------------------------------------------------------------------
// compact: with L live pages, the live pages at L and above move into the
// free ones below L, both in ascending order; afterwards the pages at L and
// above are free. No page is both read and written, so the moves need no
// order. The plan writes the two lists and the new number of each moved page.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kApplyThreads) k_pages_compact_apply(PagesParams p) {
    pdl_trigger();
    pdl_wait();
    const int32_t live = __ldcg(p.head), moves = __ldcg(p.head + 1);
    const int64_t t0 = (int64_t)blockIdx.x * kApplyThreads + threadIdx.x, step = (int64_t)gridDim.x * kApplyThreads;
    for (int64_t r = t0; r < moves; r += step) {
        const int32_t a = __ldcg(p.copy_src + r);
        p.refs[__ldcg(p.copy_dst + r)] = p.refs[a];
        p.refs[a] = 0;
    }
    // a sequence's pages end with its length; what lies behind is left alone. A
    // warp takes kRowPiece columns of a row at a time.
    constexpr int kRowPiece = 128;
    const int32_t width = p.kv.max_pages, lane = threadIdx.x & 31;
    const int64_t pieces = ((int64_t)width + kRowPiece - 1) / kRowPiece;
    for (int64_t u = t0 >> 5; u < p.kv.batch * pieces; u += step >> 5) {
        const int64_t b = u / pieces, c0 = (u - b * pieces) * kRowPiece + lane;
        int32_t *row = p.table + b * width;
        int32_t page[kRowPiece / 32];
#pragma unroll
        for (int j = 0; j < kRowPiece / 32; ++j) page[j] = c0 + 32 * j < width ? row[c0 + 32 * j] : 0;
        const int32_t held = pages_of(max(0, p.seq_len[b]), p.kv.page_size);
#pragma unroll
        for (int j = 0; j < kRowPiece / 32; ++j) {
            const int64_t c = c0 + 32 * j;
            if (c >= min(held, width) || (page[j] >= 0 && page[j] < live)) continue;
            if (page[j] < 0 || page[j] >= p.num_pages) set_error(CSA2_DEVERR_BAD_ROW);
            else row[c] = __ldcg(p.fresh + page[j]);
        }
    }
    copy_pages(p.kv, p.copy_src, p.copy_dst, moves, p.num_pages);
}

__global__ void __launch_bounds__(kPlanThreads) k_pages_compact_plan(PagesParams p) {
    __shared__ PlanShared sh;
    const uint32_t rank = cluster_rank();
    pdl_trigger();
    pdl_wait();
    const int32_t run = ((p.num_pages + kPlanCtas - 1) / kPlanCtas + 3) & ~3;
    const int32_t lo = min((int64_t)p.num_pages, (int64_t)rank * run), hi = min((int64_t)p.num_pages, (int64_t)lo + run);
    const int32_t rounds = (hi - lo + 4 * kPlanThreads - 1) / (4 * kPlanThreads);
    int32_t mine = 0;
    uint32_t total;
    for (int32_t k = 0; k < rounds; ++k) {
        const int4 r = plan_refs(p.refs, plan_page(lo, k), hi);
        mine += (r.x > 0) + (r.y > 0) + (r.z > 0) + (r.w > 0);
    }
    block_exclusive(mine, sh.warp_sums, total);
    if (threadIdx.x == 0) sh.count[0] = (int32_t)total;
    cluster_sync_all();
    int32_t live_before, live;
    cluster_sums(sh, 0, rank, live_before, live);
    // live pages at or above L before page x: live below x less the live below
    // L; holes below L before x: x less the live below x. Both follow from the
    // live count below this run and, for L, from the number of holes.
    mine = 0;
    for (int32_t k = 0; k < rounds; ++k) {
        const int32_t page = plan_page(lo, k);
        const int4 r = plan_refs(p.refs, page, hi);
        const int32_t v[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) mine += page + j < min(hi, live) && v[j] <= 0;
    }
    block_exclusive(mine, sh.warp_sums, total);
    if (threadIdx.x == 0) sh.count[1] = (int32_t)total;
    cluster_sync_all();
    int32_t hole_before, holes;
    cluster_sums(sh, 1, rank, hole_before, holes);
    const int32_t low = live - holes;  // live pages below L
    int32_t before = live_before;
    for (int32_t k = 0; k < rounds; ++k) {
        const int32_t page = plan_page(lo, k);
        const int4 r = plan_refs(p.refs, page, hi);
        const int32_t v[4] = {r.x, r.y, r.z, r.w};
        uint32_t t;
        int32_t at = before + block_exclusive((v[0] > 0) + (v[1] > 0) + (v[2] > 0) + (v[3] > 0), sh.warp_sums, t);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int32_t x = page + j;  // at: live pages below x
            if (x >= hi) break;
            if (v[j] > 0) {
                if (x >= live) p.copy_src[at - low] = x;
                ++at;
            } else if (x < live) {
                p.copy_dst[x - at] = x;
            } else {
                p.fresh[x] = x;  // free and staying so: a table that names it all the same keeps its number
            }
        }
        before += t;
    }
    const int32_t cap = p.num_pages / 2;
    for (int32_t r = holes + rank * kPlanThreads + threadIdx.x; r < cap; r += kPlanCtas * kPlanThreads)
        p.copy_src[r] = p.copy_dst[r] = -1;
    if (rank == 0 && threadIdx.x == 0) {
        p.head[0] = live;
        p.head[1] = holes;
        if (p.n_live) *p.n_live = live;
    }
    cluster_sync_all();  // both lists are in place
    for (int32_t r = rank * kPlanThreads + threadIdx.x; r < holes; r += kPlanCtas * kPlanThreads)
        p.fresh[__ldcg(p.copy_src + r)] = __ldcg(p.copy_dst + r);
}

}  // namespace csa2
