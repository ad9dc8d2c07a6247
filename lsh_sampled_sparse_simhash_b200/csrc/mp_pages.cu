// Operations on the pages of a paged key-value cache (include/magicpig.h).
//
// The state is a page table and one reference count per page; a page is free
// iff its count is 0, so there is no free list to keep in order: "the lowest
// free pages" are the zeros of the counts in index order, found by a scan.
// A plan (reserve, fork, compact) runs as ONE cluster of kPlanBlocks blocks:
// each warp owns a contiguous run of pages, counts its free (or used) ones,
// the counts meet in distributed shared memory, and a second walk over the
// run knows every page's rank.  Whole numbers only, no order that depends on
// timing: the same call always takes the same pages.
//
// The plans move a few hundred kilobytes at most and are bound by latency
// (dependent loads and cluster barriers): ending 40 of 256 sequences and
// reserving for the rest takes 15 us with 124k pages and 1000 columns, a
// compaction plan of 2900 pages 9 us.  Past 131072 pages a warp's run no longer
// fits its registers and the second walk reads the counts again, 32 at a time:
// reserve 10.5 us at 131072 pages, 17 at 131073, 26 at 2^20; compact, half of
// the pages in use and half of those to be moved, 41, 56 and 349 us.  A cluster,
// and not more blocks, because
// its barrier costs under a microsecond while a second launch costs two.  The
// page copies and the append are bound by HBM: 88 MB in 13 us (6.7 TB/s), 196
// MB of a strided projection's rows in 28.5 us (6.9 TB/s).  Loads of the counts
// bypass L1 (ld.global.cg): other blocks of the cluster change them between two
// barriers.
#include <cooperative_groups.h>

#include "mp_pages.cuh"

namespace mp {
namespace cg = cooperative_groups;

constexpr int kPlanBlocks = 8;    // portable cluster size
constexpr int kPlanThreads = 512;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanUnroll = 16;   // 32-page groups in flight per warp

// ---------------------------------------------------------- plan helpers ----
// The run of pages [lo, hi) of one warp of the cluster; runs are whole groups
// of 32 pages, in (block, warp) order.
struct PageRun {
    int lo, hi;
};
__device__ __forceinline__ int run_groups(int P)
{
    return ((P + 31) / 32 + kPlanBlocks * kPlanWarps - 1) / (kPlanBlocks * kPlanWarps);
}
__device__ __forceinline__ PageRun page_run(int P, int block, int warp)
{
    const int groups = (P + 31) / 32, per = run_groups(P);
    const int g = (block * kPlanWarps + warp) * per;
    PageRun r;
    r.lo = min(g, groups) * 32;
    r.hi = min(min(g + per, groups) * 32, P);
    return r;
}

// Used pages (count > 0) of a run.  word: lane g keeps the used bits of the
// run's g-th group of 32 (the first 32 groups), so that a run of up to 1024
// pages (a pool of up to 131072) is read once.
__device__ __forceinline__ int count_used(const int32_t *refs, PageRun r, int lane, uint32_t &word)
{
    int n = 0, g = 0;
    word = 0u;
    for (int p0 = r.lo; p0 < r.hi; p0 += 32 * kPlanUnroll) {
        int v[kPlanUnroll];
#pragma unroll
        for (int j = 0; j < kPlanUnroll; j++) {
            const int p = p0 + 32 * j + lane;
            v[j] = p < r.hi ? __ldcg(refs + p) : 0;
        }
#pragma unroll
        for (int j = 0; j < kPlanUnroll; j++, g++) {
            const uint32_t used = __ballot_sync(0xffffffffu, v[j] > 0);
            n += __popc(used);
            if (lane == g) word = used;
        }
    }
    return n;
}

// Calls f(page, in the run?, used?, used pages before it) for the pages of the
// run, all lanes of a 32-page group together; f returns false (uniformly) to
// stop.  Pages below `from` are not looked at (used_before covers them).
template <typename F>
__device__ __forceinline__ void walk_pages(const int32_t *refs, PageRun r, uint32_t word, int from, int used_before, int lane,
                                           F f)
{
    const bool kept = r.hi - r.lo <= 1024;
    int before = used_before;
    for (int p0 = r.lo, g = 0; p0 < r.hi; p0 += 32, g++) {
        const int p = p0 + lane;
        uint32_t used = kept ? __shfl_sync(0xffffffffu, word, g)
                             : __ballot_sync(0xffffffffu, p < r.hi && __ldcg(refs + p) > 0);
        if (p0 < from) used &= from - p0 >= 32 ? 0u : ~0u << (from - p0);
        if (!f(p, p >= from && p < r.hi, (used >> lane) & 1u, before + __popc(used & ((1u << lane) - 1u)))) return;
        before += __popc(used);
    }
}

// Calls f(page, rank) for the free pages with rank < total (rank: free pages
// before it) of a block's runs, its groups of 32 pages dealt out over its
// warps: the lowest free pages often lie in the runs of one or two.
template <typename F>
__device__ __forceinline__ void take_pages(const int32_t *refs, int P, PageRun r, uint32_t word, int used_before, int total,
                                           int warp, int lane, F f)
{
    __shared__ uint32_t words[kPlanWarps][32];
    __shared__ int first[kPlanWarps][32], lo[kPlanWarps], kept[kPlanWarps];
    int pre = __popc(word);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, pre, o);
        if (lane >= o) pre += x;
    }
    words[warp][lane] = word;
    first[warp][lane] = r.lo + 32 * lane - (used_before + pre - __popc(word));  // rank of the group's first free page
    if (lane == 0) {
        lo[warp] = r.lo;
        kept[warp] = r.hi - r.lo <= 1024 ? r.hi : -1;
    }
    __syncthreads();
    const int groups = min(run_groups(P), 32);
    for (int g = 0; g < groups; g++) {  // another run for every group
        const int w = (warp + g) % kPlanWarps, p = lo[w] + 32 * g + lane;
        if (kept[w] < 0 || lo[w] + 32 * g >= kept[w] || first[w][g] >= total) continue;
        const uint32_t is_free = ~words[w][g];
        const int k = first[w][g] + __popc(is_free & ((1u << lane) - 1u));
        if (p < kept[w] && ((is_free >> lane) & 1u) && k < total) f(p, k);
    }
    if (r.hi - r.lo > 1024)  // a run too long for its words: walked by its own warp
        walk_pages(refs, r, word, 0, used_before, lane, [&](int p, bool in, bool used_page, int before) {
            const int k = p - before;
            if (in && !used_page && k < total) f(p, k);
            return __any_sync(0xffffffffu, k < total);
        });
}

// Shared state of a plan.
struct PlanShared {
    int used[kPlanBlocks];   // used pages of every block's runs
    int flag[kPlanBlocks];   // every block's error code (0: none)
    int lru;                 // compact: used pages below U
    int warp_used[kPlanWarps];
    int scan[kPlanWarps];
};

// Used pages before this warp's run, and in all; the block's error code is
// spread with the same barrier, and the first one found is returned.
__device__ __forceinline__ int plan_meet(PlanShared &sh, int used_warp, int err, int &before, int &total)
{
    cg::cluster_group cl = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, blk = (int)cl.block_rank();
    err = __syncthreads_or(err != 0) ? err : 0;  // a barrier for the block; below, the block's worst code
    if (tid == 0) sh.scan[0] = 0;
    if (lane == 0) sh.warp_used[warp] = used_warp;
    __syncthreads();
    if (err) atomicMin(&sh.scan[0], err);
    __syncthreads();
    if (tid < kPlanBlocks) {
        int n = 0;
        for (int w = 0; w < kPlanWarps; w++) n += sh.warp_used[w];
        *cl.map_shared_rank(&sh.used[blk], tid) = n;
        *cl.map_shared_rank(&sh.flag[blk], tid) = sh.scan[0];
    }
    cl.sync();
    before = total = 0;
    int first = 0;
    for (int b = 0; b < kPlanBlocks; b++) {
        if (b < blk) before += sh.used[b];
        total += sh.used[b];
        first = min(first, sh.flag[b]);
    }
    for (int w = 0; w < warp; w++) before += sh.warp_used[w];
    return first;
}

// Exclusive prefix sums of a[0 .. n) in place (n <= kPagesMaxBatch); returns
// the total.  64-bit, so that no sum wraps; a total past 2^30 comes back as
// 2^30 (then nothing is taken and the prefixes are not used).
__device__ __forceinline__ int block_exclusive(int *a, int n, PlanShared &sh)
{
    constexpr int kPer = kPagesMaxBatch / kPlanThreads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    long long v[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; i++) {
        const int j = tid * kPer + i;
        v[i] = j < n ? a[j] : 0;
        sum += v[i];
    }
    long long pre = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, pre, o);
        if (lane >= o) pre += x;
    }
    const int cap = 1 << 30;
    __syncthreads();
    if (lane == 31) sh.scan[warp] = (int)min(pre, (long long)cap);
    __syncthreads();
    long long off = 0, total = 0;
    for (int w = 0; w < kPlanWarps; w++) {
        if (w < warp) off += sh.scan[w];
        total += sh.scan[w];
    }
    pre += off - sum;
#pragma unroll
    for (int i = 0; i < kPer; i++) {
        const int j = tid * kPer + i;
        if (j < n) a[j] = (int)min(pre, (long long)cap);
        pre += v[i];
    }
    __syncthreads();
    return (int)min(total, (long long)cap);
}

// The last i in [0, n) with pre[i] <= k (pre[0] = 0, not decreasing).
__device__ __forceinline__ int find_slot(const int *pre, int n, int k)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= k) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Pages that a table row holds: its leading entries >= 0.  A 17-ary search by
// half a warp (so two rows a warp, and three dependent loads for 4000
// columns); row is null for a half without one.
__device__ __forceinline__ int held_pages(const int32_t *row, int M, int lane)
{
    const int sub = lane & 15, shift = lane & 16;
    int lo = 0, hi = row ? M : 0;  // row[lo - 1] >= 0 (or lo = 0), row[hi] < 0 (or hi = M)
    while (__any_sync(0xffffffffu, lo < hi)) {
        const int step = max((hi - lo + 15) / 16, 1), at = lo + step * sub;
        const bool held = at < hi && __ldcg(row + at) >= 0;
        const unsigned bal = (__ballot_sync(0xffffffffu, held) >> shift) & 0xffffu;
        const int k = __ffs((int)~bal) - 1;  // leading probes that hold a page (16: all)
        if (lo < hi) {
            if (k == 0) {
                hi = lo;
            } else {
                const int end = lo + step * k;
                lo += step * (k - 1) + 1;
                hi = min(hi, end);
            }
        }
    }
    return lo;
}

// --------------------------------------------------------------- reserve ----
__global__ void __cluster_dims__(kPlanBlocks, 1, 1) __launch_bounds__(kPlanThreads)
    pages_reserve_kernel(PagesShape s, const int32_t *n_new, int32_t *table, const int32_t *lens, int32_t *refs,
                         int32_t *status)
{
    __shared__ PlanShared sh;
    __shared__ int need[kPagesMaxBatch], have[kPagesMaxBatch];
    cg::cluster_group cl = cg::this_cluster();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, blk = (int)cl.block_rank();
    grid_dependency_wait();
    cl.sync();  // every block of the cluster runs before its shared memory is written from another
    int err = 0;
    const PageRun run = page_run(s.P, blk, warp);
    uint32_t word;
    const int mine = count_used(refs, run, lane, word);
    for (int b0 = 2 * (blk * kPlanWarps + warp); b0 < s.B; b0 += 2 * kPlanBlocks * kPlanWarps) {  // two rows a warp
        const int b = b0 + (lane >> 4);
        const bool in = b < s.B;
        const int n = in ? n_new[b] : 0, len = in ? lens[b] : 0;
        const int h = held_pages(in ? table + (size_t)b * s.M : nullptr, s.M, lane);
        long long want = 0;
        if (n > 0) {
            const long long all = (long long)max(len, 0) + n;
            if (len < 0 || all > (long long)s.M * s.S) err = MP_ERR_CAPACITY;
            else want = max((all + s.S - 1) / s.S - h, 0ll);
        }
        if (in && (lane & 15) < kPlanBlocks) {
            *cl.map_shared_rank(&need[b], lane & 15) = (int)want;
            *cl.map_shared_rank(&have[b], lane & 15) = h;
        }
    }
    int before, used;
    err = plan_meet(sh, mine, err, before, used);
    const int total = block_exclusive(need, s.B, sh);
    if (total > s.P - used && !err) err = MP_ERR_CAPACITY;
    if (err) {
        if (blk == 0 && threadIdx.x == 0) set_status(status, err);
        return;
    }
    take_pages(refs, s.P, run, word, before, total, warp, lane, [&](int p, int k) {
        const int b = find_slot(need, s.B, k);
        table[(size_t)b * s.M + have[b] + (k - need[b])] = p;
        refs[p] = 1;
    });
}

// ------------------------------------------------------------------ fork ----
__global__ void __cluster_dims__(kPlanBlocks, 1, 1) __launch_bounds__(kPlanThreads)
    pages_fork_kernel(PagesShape s, const int32_t *src, const int32_t *dst, int n, int32_t *table, int32_t *lens,
                      int32_t *refs, int4 *copies, int32_t *status)
{
    __shared__ PlanShared sh;
    __shared__ int need[kPagesMaxBatch];
    __shared__ unsigned char is_src[kPagesMaxBatch];
    __shared__ int is_dst[kPagesMaxBatch];
    cg::cluster_group cl = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, blk = (int)cl.block_rank();
    grid_dependency_wait();
    for (int b = tid; b < s.B; b += kPlanThreads) {
        is_src[b] = 0;
        is_dst[b] = 0;
    }
    cl.sync();
    int err = 0;
    const PageRun run = page_run(s.P, blk, warp);
    uint32_t word;
    const int mine = count_used(refs, run, lane, word);
    // every block looks the whole list over
    for (int i = tid; i < n; i += kPlanThreads) {
        const int a = src[i], b = dst[i];
        int want = 0;
        if (a < 0 || a >= s.B || b < 0 || b >= s.B) {
            err = MP_ERR_ARG;
        } else {
            is_src[a] = 1;
            if (atomicAdd(&is_dst[b], 1) != 0) err = MP_ERR_ARG;
            const int len = lens[a];
            if (len < 0 || len > (long long)s.M * s.S) err = MP_ERR_ARG;
            else want = len % s.S != 0;
        }
        need[i] = want;
    }
    __syncthreads();
    // a warp per fork: the source's pages are there and in use, the row to fill is empty
    for (int i = blk * kPlanWarps + warp; i < n; i += kPlanBlocks * kPlanWarps) {
        const int a = src[i], b = dst[i];
        if (a < 0 || a >= s.B || b < 0 || b >= s.B) continue;
        if (is_src[b] || table[(size_t)b * s.M] >= 0) err = MP_ERR_ARG;
        const int len = lens[a];
        if (len < 0 || len > (long long)s.M * s.S) continue;
        const int np = (int)(((long long)len + s.S - 1) / s.S);
        for (int c = lane; c < np; c += 32) {
            const int p = table[(size_t)a * s.M + c];
            if (p < 0 || p >= s.P || __ldcg(refs + p) < 1) err = MP_ERR_ARG;
        }
    }
    int before, used;
    err = plan_meet(sh, mine, err, before, used);
    const int total = block_exclusive(need, n, sh);
    if (!err && total > s.P - used) err = MP_ERR_CAPACITY;
    if (blk == 0 && tid == 0) copies[0] = make_int4(err ? 0 : total, 0, 0, 0);
    if (err) {
        if (blk == 0 && tid == 0) set_status(status, err);
        return;
    }
    take_pages(refs, s.P, run, word, before, total, warp, lane, [&](int p, int k) {
        const int i = find_slot(need, n, k);  // the last fork with k pages before it: the one that takes this page
        const int a = src[i], len = lens[a], c = len / s.S;
        table[(size_t)dst[i] * s.M + c] = p;
        refs[p] = 1;
        copies[1 + k] = make_int4(table[(size_t)a * s.M + c], p, len % s.S, 0);
    });
    for (int i = blk * kPlanWarps + warp; i < n; i += kPlanBlocks * kPlanWarps) {
        const int a = src[i], b = dst[i], len = lens[a], full = len / s.S, keep = full + (len % s.S != 0);
        for (int c = lane; c < s.M; c += 32) {
            if (c < full) {
                const int p = table[(size_t)a * s.M + c];
                table[(size_t)b * s.M + c] = p;
                atomicAdd(refs + p, 1);
            } else if (c >= keep) {
                table[(size_t)b * s.M + c] = -1;
            }
        }
        if (lane == 0) lens[b] = len;
    }
}

// ------------------------------------------------------------------ free ----
// One block per entry of the list.  Only the first entry of a sequence acts.
constexpr int kFreeThreads = 256, kFreeBatch = 4;

__global__ void __launch_bounds__(kFreeThreads) pages_free_kernel(PagesShape s, const int32_t *seqs, int32_t *table, int32_t *lens,
                                                         int32_t *refs, int32_t *status)
{
    grid_dependency_wait();
    const int i = blockIdx.x, b = seqs[i];
    if (b < 0 || b >= s.B) {
        if (threadIdx.x == 0) set_status(status, MP_ERR_ARG);
        return;
    }
    int again = 0;
    for (int j = threadIdx.x; j < i; j += blockDim.x) again |= seqs[j] == b;
    if (__syncthreads_or(again)) return;
    int32_t *row = table + (size_t)b * s.M;
    for (int c0 = 0; c0 < s.M; c0 += kFreeThreads * kFreeBatch) {  // loads, then counts, in batches: both are round trips
        int p[kFreeBatch], old[kFreeBatch];
#pragma unroll
        for (int j = 0; j < kFreeBatch; j++) {
            const int c = c0 + j * kFreeThreads + threadIdx.x;
            p[j] = c < s.M ? row[c] : -1;
        }
#pragma unroll
        for (int j = 0; j < kFreeBatch; j++) old[j] = p[j] >= 0 && p[j] < s.P ? atomicSub(refs + p[j], 1) : 1;
#pragma unroll
        for (int j = 0; j < kFreeBatch; j++) {
            if (p[j] < 0) continue;
            if (p[j] >= s.P || old[j] <= 0) {
                if (p[j] < s.P) atomicAdd(refs + p[j], 1);
                set_status(status, MP_ERR_ARG);
            }
            row[c0 + j * kFreeThreads + threadIdx.x] = -1;
        }
    }
    if (threadIdx.x == 0) lens[b] = 0;
}

// --------------------------------------------------------------- compact ----
__global__ void __cluster_dims__(kPlanBlocks, 1, 1) __launch_bounds__(kPlanThreads)
    pages_compact_kernel(PagesShape s, int32_t *table, int32_t *refs, int32_t *copies, int32_t *status)
{
    __shared__ PlanShared sh;
    cg::cluster_group cl = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, blk = (int)cl.block_rank();
    grid_dependency_wait();
    cl.sync();
    const PageRun run = page_run(s.P, blk, warp);
    uint32_t word;
    const int mine = count_used(refs, run, lane, word);
    int before, U;
    plan_meet(sh, mine, 0, before, U);
    // the i-th free page below U takes move i; whoever meets page U tells all how many used ones are below it
    walk_pages(refs, run, word, 0, before, lane, [&](int p, bool in, bool used_page, int used_before) {
        if (in && p < U && !used_page) copies[4 * (1 + p - used_before) + 1] = p;
        if (in && p == U)
            for (int b = 0; b < kPlanBlocks; b++) *cl.map_shared_rank(&sh.lru, b) = used_before;
        return __any_sync(0xffffffffu, in && p <= U);
    });
    cl.sync();
    const int lru = U < s.P ? sh.lru : U;  // U - lru pages move
    if (blk == 0 && tid == 0) {
        copies[0] = U - lru;
        copies[1] = copies[2] = copies[3] = 0;
    }
    if (U == lru) return;  // the same for all blocks
    // the pages from U on move (those below are being given counts meanwhile)
    walk_pages(refs, run, word, U, run.lo > U ? before : lru, lane, [&](int p, bool in, bool used_page, int used_before) {
        if (in && used_page) {
            int32_t *e = copies + 4 * (size_t)(1 + used_before - lru);
            const int to = __ldcg(e + 1);
            e[0] = p;
            e[2] = s.S;
            e[3] = 0;
            refs[to] = __ldcg(refs + p);
            refs[p] = -1 - to;  // where it went, until the table has followed
        }
        return true;
    });
    cl.sync();
    const size_t entries = (size_t)s.B * s.M;
    for (size_t i = (size_t)blk * kPlanThreads + tid; i < entries; i += (size_t)kPlanBlocks * kPlanThreads) {
        const int p = table[i];
        if (p >= U && p < s.P) {
            const int r = __ldcg(refs + p);
            if (r < 0) table[i] = -1 - r;
        }
    }
    cl.sync();
    for (int p = max(run.lo, U) + lane; p < run.hi; p += 32)
        if (__ldcg(refs + p) < 0) refs[p] = 0;
}

// ------------------------------------------------------------------ copy ----
// A warp moves kCopyRows rows of one head of one page (4 KB, one 16-byte piece
// of every row pair per lane and step), all its loads before its stores, so a
// full SM has 256 KB in flight.
constexpr int kCopyRows = 16;
constexpr int kCopyWarps = 8;

__global__ void __launch_bounds__(32 * kCopyWarps) pages_copy_kernel(PagesShape s, const int4 *copies, int max_copies,
                                                                    uint4 *kp, uint4 *vp, int32_t *status)
{
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    int n = copies[0].x;
    if (n < 0 || n > max_copies) {
        if (blockIdx.x == 0 && threadIdx.x == 0) set_status(status, MP_ERR_ARG);
        n = min(max(n, 0), max_copies);
    }
    const int segs = (s.S + kCopyRows - 1) / kCopyRows;
    const long long per = 2ll * s.Hkv * segs, units = per * n;
    const long long stride = (long long)gridDim.x * kCopyWarps;
    for (long long u = (long long)blockIdx.x * kCopyWarps + (threadIdx.x >> 5); u < units; u += stride) {
        const int4 e = copies[1 + u / per];
        int rest = (int)(u % per);
        const int seg = rest % segs;
        rest /= segs;
        const int h = rest >> 1, row0 = seg * kCopyRows;
        if (e.x < 0 || e.x >= s.P || e.y < 0 || e.y >= s.P || e.z < 0 || e.z > s.S) {
            if (lane == 0) set_status(status, MP_ERR_ARG);
            continue;
        }
        const int pieces = min(e.z - row0, kCopyRows) * (kHeadDim / 8);
        if (pieces <= 0) continue;
        uint4 *pool = (rest & 1) ? vp : kp;
        const uint4 *from = pool + (((size_t)e.x * s.Hkv + h) * s.S + row0) * (kHeadDim / 8);
        uint4 *to = pool + (((size_t)e.y * s.Hkv + h) * s.S + row0) * (kHeadDim / 8);
        uint4 v[kCopyRows / 2];
#pragma unroll
        for (int j = 0; j < kCopyRows / 2; j++)
            if (32 * j + lane < pieces) v[j] = __ldcs(from + 32 * j + lane);
#pragma unroll
        for (int j = 0; j < kCopyRows / 2; j++)
            if (32 * j + lane < pieces) to[32 * j + lane] = v[j];
    }
}

// ---------------------------------------------------------------- append ----
// A warp per new token row: it finds its sequence, position and page, then
// moves the row's Hkv key and Hkv value vectors, kAppendBatch pieces in flight
// per lane.  Bound by HBM (each row read once and written once); for one
// token a sequence by latency.
constexpr int kAppendWarps = 8;
constexpr int kAppendBatch = 8;

// The sequence of row r: the last b in [0, B) with cu[b] <= r.
__device__ __forceinline__ int find_sequence(const int32_t *cu, int B, int r, int lane)
{
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + step * lane;
        const unsigned bal = __ballot_sync(0xffffffffu, at < hi && cu[at] <= r);
        const int k = max(bal == 0xffffffffu ? 32 : __ffs((int)~bal) - 1, 1);
        hi = min(hi, lo + step * k);
        lo = lo + step * (k - 1);
    }
    return lo;
}

__device__ __forceinline__ bool bad_range(int lo, int hi, int total) { return lo < 0 || hi < lo || hi > total; }

__global__ void __launch_bounds__(32 * kAppendWarps) paged_append_kernel(PagesShape s, const uint16_t *k_new,
                                                                        const uint16_t *v_new, int64_t ks, int64_t vs,
                                                                        const int32_t *cu, int n_rows, int advance,
                                                                        const int32_t *table, int32_t *lens, uint4 *kp,
                                                                        uint4 *vp, int32_t *status)
{
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    if (cu && blockIdx.x == 0)
        for (int b = threadIdx.x; b < s.B; b += blockDim.x)
            if (bad_range(cu[b], cu[b + 1], n_rows)) set_status(status, MP_ERR_CAPACITY);
    const int r = blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
    if (r >= n_rows) return;
    int b = r, i = 0;
    if (cu) {
        b = find_sequence(cu, s.B, r, lane);
        const int lo = cu[b], hi = cu[b + 1];
        if (bad_range(lo, hi, n_rows) || r < lo || r >= hi) return;  // a row of no sequence
        i = r - lo;
    }
    const int len = lens[b];
    const long long pos = (long long)len + i;
    const bool room = len >= 0 && pos < (long long)s.M * s.S;
    const int page = room ? table[(size_t)b * s.M + pos / s.S] : -1;
    if (page < 0 || page >= s.P) {
        if (lane == 0) set_status(status, MP_ERR_CAPACITY);
        return;
    }
    constexpr int kPieces = kHeadDim / 8;  // 16-byte pieces of a vector
    const size_t dst0 = ((size_t)page * s.Hkv * s.S + pos % s.S) * kPieces;
    const uint4 *kr = reinterpret_cast<const uint4 *>(k_new + (size_t)r * ks);
    const uint4 *vr = reinterpret_cast<const uint4 *>(v_new + (size_t)r * vs);
    const int half = s.Hkv * kPieces;  // pieces of the row's keys (then as many of its values)
    for (int p0 = 0; p0 < 2 * half; p0 += 32 * kAppendBatch) {
        uint4 x[kAppendBatch];
#pragma unroll
        for (int j = 0; j < kAppendBatch; j++) {
            const int p = p0 + 32 * j + lane;
            if (p < 2 * half) x[j] = __ldcs(p < half ? kr + p : vr + (p - half));
        }
#pragma unroll
        for (int j = 0; j < kAppendBatch; j++) {
            const int p = p0 + 32 * j + lane;
            if (p < 2 * half) {
                const int e = p < half ? p : p - half;
                (p < half ? kp : vp)[dst0 + (size_t)(e / kPieces) * s.S * kPieces + e % kPieces] = x[j];
            }
        }
    }
    if (!cu && advance) {
        __syncwarp();  // every lane has read the length
        if (lane == 0) lens[b] = len + 1;  // this warp alone reads and writes it
    }
}

// Moves the lengths after a packed append (its own launch: every row of a
// sequence reads the old length).  A warp per sequence; a sequence that lacks
// a page for one of its rows keeps its length, and all do if an entry of cu
// breaks the order (rows that two sequences claim went to one of them).
__global__ void __launch_bounds__(128) paged_advance_kernel(PagesShape s, const int32_t *cu, int n_rows,
                                                            const int32_t *table, int32_t *lens)
{
    grid_dependency_wait();
    const int lane = threadIdx.x & 31, b = blockIdx.x * 4 + (threadIdx.x >> 5);
    int bad = 0;
    for (int j = threadIdx.x; j < s.B; j += blockDim.x) bad |= bad_range(cu[j], cu[j + 1], n_rows);
    if (__syncthreads_or(bad) || b >= s.B) return;
    const int lo = cu[b], hi = cu[b + 1], len = lens[b];
    if (hi == lo || len < 0) return;
    const long long end = (long long)len + (hi - lo);
    if (end > (long long)s.M * s.S) return;
    bool ok = true;
    for (int c = len / s.S + lane; c <= (int)((end - 1) / s.S); c += 32) {
        const int p = table[(size_t)b * s.M + c];
        ok = ok && p >= 0 && p < s.P;
    }
    if (__all_sync(0xffffffffu, ok) && lane == 0) lens[b] = (int)end;
}

// ------------------------------------------------------------------ host ----
cudaError_t launch_pages_reserve(const PagesShape &s, const int32_t *n_new, int32_t *table, const int32_t *lens,
                                 int32_t *refs, int32_t *status, cudaStream_t st)
{
    return launch_pdl(pages_reserve_kernel, dim3(kPlanBlocks), dim3(kPlanThreads), 0, st, s, n_new, table, lens, refs,
                      status);
}

cudaError_t launch_pages_fork(const PagesShape &s, const int32_t *src, const int32_t *dst, int n, int32_t *table,
                              int32_t *lens, int32_t *refs, int32_t *copies, int32_t *status, cudaStream_t st)
{
    return launch_pdl(pages_fork_kernel, dim3(kPlanBlocks), dim3(kPlanThreads), 0, st, s, src, dst, n, table, lens, refs,
                      reinterpret_cast<int4 *>(copies), status);
}

cudaError_t launch_pages_free(const PagesShape &s, const int32_t *seqs, int n, int32_t *table, int32_t *lens,
                              int32_t *refs, int32_t *status, cudaStream_t st)
{
    return launch_pdl(pages_free_kernel, dim3(n), dim3(kFreeThreads), 0, st, s, seqs, table, lens, refs, status);
}

cudaError_t launch_pages_compact(const PagesShape &s, int32_t *table, int32_t *refs, int32_t *copies, int32_t *status,
                                 cudaStream_t st)
{
    return launch_pdl(pages_compact_kernel, dim3(kPlanBlocks), dim3(kPlanThreads), 0, st, s, table, refs, copies, status);
}

cudaError_t launch_pages_copy(const PagesShape &s, const int32_t *copies, int max_copies, uint16_t *kp, uint16_t *vp,
                              int32_t *status, cudaStream_t st)
{
    if (max_copies == 0) return cudaSuccess;
    const long long segs = (s.S + kCopyRows - 1) / kCopyRows;
    const long long units = 2ll * s.Hkv * segs * max_copies;
    const long long blocks = (units + kCopyWarps - 1) / kCopyWarps;
    const int grid = (int)(blocks < 148 * 8 ? blocks : 148 * 8);  // 8 blocks of 8 warps fill an SM
    return launch_pdl(pages_copy_kernel, dim3(grid), dim3(32 * kCopyWarps), 0, st, s,
                      reinterpret_cast<const int4 *>(copies), max_copies, reinterpret_cast<uint4 *>(kp),
                      reinterpret_cast<uint4 *>(vp), status);
}

cudaError_t launch_paged_append(const PagesShape &s, const uint16_t *k_new, const uint16_t *v_new, int64_t ks, int64_t vs,
                                const int32_t *cu_new, int n_rows, int advance, const int32_t *table, int32_t *lens,
                                uint16_t *kp, uint16_t *vp, int32_t *status, cudaStream_t st)
{
    if (n_rows == 0) return cudaSuccess;
    const int grid = (n_rows + kAppendWarps - 1) / kAppendWarps;
    cudaError_t e = launch_pdl(paged_append_kernel, dim3(grid), dim3(32 * kAppendWarps), 0, st, s, k_new, v_new, ks, vs,
                               cu_new, n_rows, advance, table, lens, reinterpret_cast<uint4 *>(kp),
                               reinterpret_cast<uint4 *>(vp), status);
    if (e == cudaSuccess && cu_new && advance)
        e = launch_pdl(paged_advance_kernel, dim3((s.B + 3) / 4), dim3(128), 0, st, s, cu_new, n_rows, table,
                       (int32_t *)lens);
    return e;
}

}  // namespace mp
