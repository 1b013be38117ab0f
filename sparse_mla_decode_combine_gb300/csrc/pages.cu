// pages.cu -- operators on the pages of a paged cache: forking rows (with copy-on-write of their
// last page, or private copies), compacting the live pages to the front of the pool, and copying
// listed pages.  They move whole entries and never look into them, so any entry format will do.
//
// The pool's state is three arrays: the block table, the rows' lengths, and a reference count per
// page (0: the page is free).  New pages are the lowest-numbered free ones, so the result of a call
// depends on its inputs alone; integer sums are the only atomics.
//
// Every operator is two launches: a planning kernel does the index work (counts, ranks and sums over the
// reference counts and rows) and writes which pages are copied where; a second kernel over the whole GPU
// moves the pages of every layer.  The second is bound by HBM (each byte read and written once), the first by
// the latency of its dependent steps, so it takes as few trips to global memory as it can: in a pool of up to
// 16384 pages one CTA does it, with the counts, the rows' numbers and the free list in shared memory; larger
// ones take a cluster of eight CTAs with a cluster barrier between the steps and the numbers in the workspace,
// and so do forks of many rows or wide tables, whose cells 32 warps read too slowly.  A compaction that moves
// 418 MB takes 140 us where the bytes alone take 123 at the measured 6794 GB/s.
// A short list of pages to copy needs no plan: one launch.
#include <algorithm>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fp4.h"

namespace dsv4 {
namespace {

constexpr int kCluster = 8;
constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kCluster * kPlanThreads / 32;
constexpr int kCopyThreads = 256;
constexpr int kFewSmall = 2048;        // small pages that are copied without a plan
constexpr int kCopyUnroll = 8;         // 16-byte pieces a thread holds: a page of 64 entries of 400 bytes in one round of a CTA
// The one-CTA plans, against those of eight CTAs, in us with a move of little.  Compact: 333 pages 4.8 / 8.3, 8192 pages
// 8.6 / 10.0, 12000 pages 10.3 / 11.3, 16384 pages 12.4 / 12.1.  Fork, rows x cells: of 4096 pages 64 x 64 9.2 / 13.2, 128 x 64
// 12.6 / 13.6, 160 x 64 14.3 / 13.1, 64 x 256 10.8 / 12.9, 96 x 256 13.2 / 12.8; of 16384 pages 64 x 256 15.4 / 16.5, 128 x 8
// 14.7 / 14.1, 64 x 1024 22.0 / 18.3, 1024 x 8 57 / 25.
constexpr int kSmallPages = 16384;     // pages,
constexpr int kSmallRows = 128;        // rows before and after (at most one to a thread),
constexpr int kSmallCells = 1 << 14;   // and cells of the table

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ int cluster_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return (int)r;
}

// the copy of `v` in the shared memory of the cluster's CTA `rank`
__device__ __forceinline__ int ld_rank(const int *v, int rank)
{
    uint32_t a;
    int x;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(v)), "r"(rank));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(x) : "r"(a) : "memory");
    return x;
}

// exclusive sum of v over the CTA's threads; *total receives the sum.  Two barriers.
__device__ __forceinline__ int cta_scan(int v, int *wsum, int *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d)
            x += y;
    }
    __syncthreads();   // (the previous use of wsum is over)
    if (lane == 31)
        wsum[warp] = x;
    __syncthreads();
    const int ws = wsum[lane];   // kPlanThreads / 32 = 32 warps
    int before = lane < warp ? ws : 0, all = ws;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        before += __shfl_xor_sync(0xffffffffu, before, d);
        all += __shfl_xor_sync(0xffffffffu, all, d);
    }
    *total = all;
    return before + x - v;
}

__device__ __forceinline__ int pages_of(int len, int page, int max_blocks)
{
    const int n = len <= 0 ? 0 : (len - 1) / page + 1;
    return n < max_blocks ? n : max_blocks;
}

// entries that page j of a row of `len` entries holds
__device__ __forceinline__ int entries_of(int len, int page, int j)
{
    const int64_t left = (int64_t)len - (int64_t)j * page;
    return left < page ? (int)left : page;
}

// ---- fork ----------------------------------------------------------------------------------------

// Row r of the output is a copy of row parent[r] (an empty row for a negative parent).  Page j of it is
//   shared   (the parent's page, one more reference)  when share is set and the page is full;
//   kept     (the parent's page)  otherwise, for the lowest output row of that parent, when the page
//            has that one reference on entry;
//   taken    (a free page, the parent's entries copied into it)  else.
// Free pages are those with a count of 0 on entry, lowest first, given out in order of (row, page); a
// row that needs pages past the last free one becomes an empty row and is flagged.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kPlanThreads) fork_plan_kernel(const ForkParams p)
{
    __shared__ int wsum[32];
    __shared__ int count;
    const int rank = cluster_rank(), tid = threadIdx.x, lane = tid & 31;
    const int gtid = rank * kPlanThreads + tid, gwarp = gtid >> 5;
    const int B = p.pool.num_blocks, page = p.pool.page;
    griddep_wait();
    griddep_launch();   // (the moving kernel waits for this grid itself)

    // ---- the free pages of this CTA's part of the pool, and the rows' empty counters
    const int part = (B + kCluster - 1) / kCluster;
    const int lo = min(B, rank * part), hi = min(B, lo + part);
    int mine = 0;
    for (int i = lo + tid; i < hi; i += kPlanThreads)
        mine += p.refs[i] == 0;
    int total;
    cta_scan(mine, wsum, &total);
    if (tid == 0)
        count = total;
    for (int i = gtid; i < p.rows; i += kCluster * kPlanThreads) {
        p.first[i] = INT32_MAX;
        p.kids[i] = 0;
    }
    cluster_sync();
    int free_before = 0, num_free = 0;
    for (int k = 0; k < kCluster; ++k) {
        const int v = ld_rank(&count, k);
        free_before += k < rank ? v : 0;
        num_free += v;
    }
    for (int r = gtid; r < p.rows_out; r += kCluster * kPlanThreads) {
        const int par = p.parent[r];
        if (par >= 0 && par < p.rows)
            atomicMin(&p.first[par], r);
        else if (par >= p.rows)
            atomicOr(p.status, kStatusBadIndex);
    }
    cluster_sync();

    // ---- each row's pages: shared and kept ones as they are, -2 for the ones to take, -1 past its end
    for (int r = gwarp; r < p.rows_out; r += kPlanWarps) {
        const int par = p.parent[r];
        const bool there = par >= 0 && par < p.rows;
        const int len = there ? p.lens[par] : 0;
        const int np = pages_of(len, page, p.max_blocks);
        const int full = p.share ? min(np, max(len, 0) / page) : 0;
        const bool is_first = there && p.first[par] == r;
        const int32_t *src = p.table + (int64_t)(there ? par : 0) * p.table_stride;
        int32_t *dst = p.table_out + (int64_t)r * p.table_out_stride;
        int need = 0;
        for (int j = lane; j < p.max_blocks; j += 32) {
            int v = -1;
            if (j < np) {
                v = src[j];
                if (v < 0 || v >= B) {
                    atomicOr(p.status, kStatusBadIndex);
                    v = -1;
                } else if (j >= full && !(is_first && p.refs[v] == 1)) {
                    v = -2;
                    ++need;
                }
            }
            dst[j] = v;
        }
        if (there && len > (int64_t)p.max_blocks * page && lane == 0)
            atomicOr(p.status, kStatusBadIndex);
        need = __reduce_add_sync(0xffffffffu, need);
        if (lane == 0)
            p.need[r] = need;
    }
    cluster_sync();

    // ---- where each row's new pages start in the list of free pages (CTA 0), and that list
    int need_sum = 0;
    for (int r0 = 0; r0 < p.rows_out; r0 += kPlanThreads) {
        const int r = r0 + tid;
        const int n = r < p.rows_out ? p.need[r] : 0;
        const int before = need_sum + cta_scan(n, wsum, &total);
        if (rank == 0 && r < p.rows_out)
            p.offset[r] = n > 0 && before + n > num_free ? -1 : before;   // -1: not enough pages
        need_sum = min(need_sum + total, INT32_MAX / 2);
    }
    const int wanted = min(need_sum, num_free);
    int running = free_before;
    for (int i0 = lo; i0 < hi; i0 += kPlanThreads) {
        const int i = i0 + tid;
        const int v = i < hi ? p.refs[i] : 1;
        const int at = running + cta_scan(v == 0, wsum, &total);
        if (v == 0 && at < wanted)
            p.free_list[at] = i;
        if (i < hi && p.refs_out != p.refs)
            p.refs_out[i] = v;
        running += total;
    }
    if (rank == 0 && tid == 0)
        *p.num_copies = wanted;
    // a row that got no pages leaves its share of the copy list unused
    for (int i = gtid; i < wanted; i += kCluster * kPlanThreads)
        p.copies[i] = make_int4(0, 0, 0, 0);
    cluster_sync();

    // ---- the new pages into the rows, and the copies that fill them
    for (int r = gwarp; r < p.rows_out; r += kPlanWarps) {
        const int par = p.parent[r];
        const bool there = par >= 0 && par < p.rows;
        const int off = p.offset[r];
        const bool ok = there && off >= 0;
        const int len = there ? min(p.lens[par], (int)min((int64_t)p.max_blocks * page, (int64_t)INT32_MAX)) : 0;
        if (lane == 0) {
            p.lens_out[r] = ok ? max(len, 0) : 0;
            if (there && !ok)
                atomicOr(p.status, kStatusBadIndex);
            if (ok)
                atomicAdd(&p.kids[par], 1);
        }
        int32_t *dst = p.table_out + (int64_t)r * p.table_out_stride;
        if (!ok) {
            if (there)
                for (int j = lane; j < p.max_blocks; j += 32)
                    dst[j] = -1;
            continue;
        }
        if (p.need[r] == 0)
            continue;
        const int32_t *src = p.table + (int64_t)par * p.table_stride;
        const int np = pages_of(len, page, p.max_blocks);
        int at = off;
        for (int j0 = 0; j0 < np; j0 += 32) {
            const int j = j0 + lane;
            const bool take = j < np && dst[j] == -2;
            const unsigned m = __ballot_sync(0xffffffffu, take);
            if (take) {
                const int k = at + __popc(m & ((1u << lane) - 1u));
                const int q = p.free_list[k];
                dst[j] = q;
                p.refs_out[q] = 1;
                p.copies[k] = make_int4(src[j], q, entries_of(len, page, j), 0);
            }
            at += __popc(m);
        }
    }
    cluster_sync();

    // ---- the old rows' references go, their children's come (a full page of a row with c children
    // changes by c - 1; a page that was kept does not change)
    for (int i = gwarp; i < p.rows; i += kPlanWarps) {
        const int len = p.lens[i];
        const int np = pages_of(len, page, p.max_blocks);
        const int full = p.share ? min(np, max(len, 0) / page) : 0;
        const int c = p.kids[i], f = p.first[i];
        const bool has = f != INT32_MAX && p.offset[f] >= 0;
        const int32_t *src = p.table + (int64_t)i * p.table_stride;
        const int32_t *kept = p.table_out + (int64_t)(has ? f : 0) * p.table_out_stride;
        if (len > (int64_t)p.max_blocks * page && lane == 0)   // (rows that nobody descends from are read here alone)
            atomicOr(p.status, kStatusBadIndex);
        for (int j = lane; j < np; j += 32) {
            const int v = src[j];
            if (v < 0 || v >= B) {
                atomicOr(p.status, kStatusBadIndex);
                continue;
            }
            const int d = j < full ? c - 1 : (has && kept[j] == v ? 0 : -1);
            if (d != 0)
                atomicAdd(&p.refs_out[v], d);
        }
    }
}

// The same plan by one CTA, for small pools and tables.
__global__ void __launch_bounds__(kPlanThreads) fork_plan_small_kernel(const ForkParams p)
{
    extern __shared__ int sm[];
    __shared__ int wsum[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int B = p.pool.num_blocks, page = p.pool.page, M = p.max_blocks;
    int *refs = sm, *refs_new = sm + B, *free_list = sm + 2 * B;
    int *first = sm + 3 * B, *kids = first + p.rows, *lens = kids + p.rows, *nps = lens + p.rows, *fulls = nps + p.rows;   // [rows]
    int *parent = fulls + p.rows, *off = parent + p.rows_out;                                                        // [rows_out]
    griddep_wait();
    griddep_launch();   // (the moving kernel waits for this grid itself)

    for (int i = tid; i < B; i += kPlanThreads)
        refs[i] = refs_new[i] = p.refs[i];
    for (int i = tid; i < p.rows; i += kPlanThreads) {
        first[i] = INT32_MAX;
        kids[i] = 0;
        const int len = p.lens[i];   // (the divisions are done here, a row to a thread, and not by every row's warp)
        lens[i] = len;
        nps[i] = pages_of(len, page, M);
        fulls[i] = p.share ? min(nps[i], max(len, 0) / page) : 0;
        if (len > (int64_t)M * page)
            atomicOr(p.status, kStatusBadIndex);
    }
    for (int r = tid; r < p.rows_out; r += kPlanThreads) {
        const int par = p.parent[r];
        if (par >= p.rows)
            atomicOr(p.status, kStatusBadIndex);
        parent[r] = par >= 0 && par < p.rows ? par : -1;
    }
    __syncthreads();
    for (int r = tid; r < p.rows_out; r += kPlanThreads)
        if (parent[r] >= 0)
            atomicMin(&first[parent[r]], r);
    const int per = (B + kPlanThreads - 1) / kPlanThreads | 1;   // a run of pages to a thread (odd: no bank conflicts)
    const int i0 = min(B, tid * per), i1 = min(B, i0 + per);
    int mine = 0, num_free, total;
    for (int i = i0; i < i1; ++i)
        mine += refs[i] == 0;
    int at_free = cta_scan(mine, wsum, &num_free);   // (its barriers also end the loop above)
    for (int i = i0; i < i1; ++i)
        if (refs[i] == 0)
            free_list[at_free++] = i;
    __syncthreads();

    // whether a row takes a page of its own for page j of its parent (which is v)
    auto takes = [&](int r, int par, int full, int j, int v) { return j >= full && !(first[par] == r && refs[v] == 1); };
    for (int r = warp; r < p.rows_out; r += kPlanThreads / 32) {
        const int par = parent[r];
        int need = 0;
        if (par >= 0) {
            const int np = nps[par], full = fulls[par];
            const int32_t *src = p.table + (int64_t)par * p.table_stride;
            for (int j = full + lane; j < np; j += 32) {   // (shared pages take nothing)
                const int v = src[j];
                need += v >= 0 && v < B && takes(r, par, full, j, v);
            }
            need = __reduce_add_sync(0xffffffffu, need);
        }
        if (lane == 0)
            off[r] = need;
    }
    __syncthreads();
    const int need = tid < p.rows_out ? off[tid] : 0;   // (one row to a thread: kSmallRows)
    const int before = cta_scan(need, wsum, &total);
    const int wanted = min(total, num_free);
    if (tid < p.rows_out)
        off[tid] = need > 0 && before + need > num_free ? -1 : before;
    if (tid == 0)
        *p.num_copies = wanted;
    for (int i = tid; i < wanted; i += kPlanThreads)   // (a row that gets no pages leaves its share unused)
        p.copies[i] = make_int4(0, 0, 0, 0);
    __syncthreads();

    for (int r = warp; r < p.rows_out; r += kPlanThreads / 32) {
        const int par = parent[r];
        const bool ok = par >= 0 && off[r] >= 0;
        const int len = ok ? min(lens[par], (int)min((int64_t)M * page, (int64_t)INT32_MAX)) : 0;
        const int np = ok ? nps[par] : 0, full = ok ? fulls[par] : 0;
        if (lane == 0) {
            p.lens_out[r] = max(len, 0);
            if (par >= 0 && !ok)
                atomicOr(p.status, kStatusBadIndex);
            if (ok)
                atomicAdd(&kids[par], 1);
        }
        const int32_t *src = p.table + (int64_t)max(par, 0) * p.table_stride;
        int32_t *dst = p.table_out + (int64_t)r * p.table_out_stride;
        int at = off[r];
        for (int j0 = 0; j0 < M; j0 += 32) {
            const int j = j0 + lane;
            int v = -1;
            bool take = false;
            if (j < np) {
                v = src[j];
                if (v < 0 || v >= B)
                    v = -1;
                else
                    take = takes(r, par, full, j, v);
            }
            const unsigned m = __ballot_sync(0xffffffffu, take);
            if (take) {
                const int k = at + __popc(m & ((1u << lane) - 1u)), q = free_list[k];
                p.copies[k] = make_int4(v, q, entries_of(len, page, j), 0);
                refs_new[q] = 1;
                v = q;
            }
            at += __popc(m);
            if (j < M)
                dst[j] = v;
        }
    }
    __syncthreads();
    for (int i = warp; i < p.rows; i += kPlanThreads / 32) {
        const int np = nps[i], full = fulls[i];
        const int c = kids[i], f = first[i];
        const bool has = f != INT32_MAX && off[f] >= 0;
        const int32_t *src = p.table + (int64_t)i * p.table_stride;
        for (int j = lane; j < np; j += 32) {   // (every cell of every row: bad ones are flagged here)
            const int v = src[j];
            if (v < 0 || v >= B) {
                atomicOr(p.status, kStatusBadIndex);
                continue;
            }
            const int d = j < full ? c - 1 : (has && refs[v] == 1 ? 0 : -1);   // (the first child kept it)
            if (d != 0)
                atomicAdd(&refs_new[v], d);
        }
    }
    __syncthreads();
    for (int i = tid; i < B; i += kPlanThreads)
        p.refs_out[i] = refs_new[i];
}

// ---- compact -------------------------------------------------------------------------------------

// With L live pages (count > 0), the k-th live page at or past L moves to the k-th free page below L.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kPlanThreads) compact_plan_kernel(const CompactParams p)
{
    __shared__ int wsum[32];
    __shared__ int count[2];
    const int rank = cluster_rank(), tid = threadIdx.x;
    const int B = p.pool.num_blocks;
    griddep_wait();
    griddep_launch();

    const int part = (B + kCluster - 1) / kCluster;
    const int lo = min(B, rank * part), hi = min(B, lo + part);
    int mine = 0, total;
    for (int i = lo + tid; i < hi; i += kPlanThreads)
        mine += p.refs[i] > 0;
    cta_scan(mine, wsum, &total);
    if (tid == 0)
        count[0] = total;
    cluster_sync();
    int before = 0, L = 0;
    for (int k = 0; k < kCluster; ++k) {
        const int v = ld_rank(&count[0], k);
        before += k < rank ? v : 0;
        L += v;
    }
    // the live pages below L
    mine = 0;
    for (int i = lo + tid; i < min(hi, L); i += kPlanThreads)
        mine += p.refs[i] > 0;
    cta_scan(mine, wsum, &total);
    if (tid == 0)
        count[1] = total;
    cluster_sync();
    int below = 0;
    for (int k = 0; k < kCluster; ++k)
        below += ld_rank(&count[1], k);
    const int moves = L - below;

    int running = before;
    for (int i0 = lo; i0 < hi; i0 += kPlanThreads) {
        const int i = i0 + tid;
        const int v = i < hi ? p.refs[i] : 0;
        const bool live = v > 0;
        const int r = running + cta_scan(live, wsum, &total);   // live pages before page i
        running += total;
        if (i >= hi)
            continue;
        if (live && i >= L) {
            p.copies[r - below].x = i;
        } else if (!live && i < L) {
            p.copies[i - r].y = i;
        } else if (p.refs_out != p.refs || v < 0) {
            p.refs_out[i] = live ? v : 0;
        }
        if (!(live && i >= L))
            p.page_map[i] = live ? i : -1;
    }
    if (rank == 0 && tid == 0) {
        *p.num_live = L;
        *p.num_copies = moves;
    }
    cluster_sync();
    for (int k = rank * kPlanThreads + tid; k < moves; k += kCluster * kPlanThreads) {
        const int4 c = p.copies[k];
        p.page_map[c.x] = c.y;
        p.refs_out[c.y] = p.refs[c.x];
        p.refs_out[c.x] = 0;
        p.copies[k].z = p.pool.page;
    }
}

// The same plan by one CTA, for small pools: a run of pages to a thread, so that one sum over the threads ranks them all
// (tile by tile, a sum to 1024 pages, 8192 pages took 6 us longer); what is written per page goes out through shared
// memory, in order.
__global__ void __launch_bounds__(kPlanThreads) compact_plan_small_kernel(const CompactParams p)
{
    extern __shared__ int sm[];
    __shared__ int wsum[32];
    const int tid = threadIdx.x;
    const int B = p.pool.num_blocks;
    const int per = (B + kPlanThreads - 1) / kPlanThreads | 1;   // (odd: no bank conflicts between the threads' runs)
    int *refs = sm, *map = sm + B, *src = map + B, *dst = src + (B + 1) / 2;
    griddep_wait();
    griddep_launch();
    for (int i = tid; i < B; i += kPlanThreads)
        refs[i] = p.refs[i];
    __syncthreads();
    const int i0 = min(B, tid * per), i1 = min(B, i0 + per);
    int mine = 0, L, below;
    for (int i = i0; i < i1; ++i)
        mine += refs[i] > 0;
    int r = cta_scan(mine, wsum, &L);   // live pages before this thread's
    mine = 0;
    for (int i = i0; i < min(i1, L); ++i)
        mine += refs[i] > 0;
    cta_scan(mine, wsum, &below);
    const int moves = L - below;
    for (int i = i0; i < i1; ++i) {
        const bool live = refs[i] > 0;
        map[i] = live ? i : -1;
        if (live && i >= L)
            src[r - below] = i;
        else if (!live && i < L)
            dst[i - r] = i;
        r += live;
    }
    if (tid == 0) {
        *p.num_live = L;
        *p.num_copies = moves;
    }
    __syncthreads();
    for (int k = tid; k < moves; k += kPlanThreads) {
        const int from = src[k], to = dst[k];
        p.copies[k] = make_int4(from, to, p.pool.page, 0);
        map[from] = to;
        refs[to] = refs[from];   // (a free page's count, and a live one's past L: each has one reader and one writer)
        refs[from] = 0;
    }
    __syncthreads();
    for (int i = tid; i < B; i += kPlanThreads) {
        p.page_map[i] = map[i];
        p.refs_out[i] = max(refs[i], 0);
    }
}

// ---- copies of listed pages ----------------------------------------------------------------------

// A target that is listed twice receives its last pair.  In one pool, a pair whose source is also a
// target of the call is refused (the page might be read before or after it is written).  Long lists are
// checked through a claim on each target; short ones (launch_copy_pages) by the moving kernel itself, a pair to a thread.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kPlanThreads) copy_plan_kernel(const CopyPagesParams p)
{
    const int gtid = cluster_rank() * kPlanThreads + threadIdx.x;
    constexpr int kStep = kCluster * kPlanThreads;
    griddep_wait();
    griddep_launch();
    auto good = [&](int s, int d) { return s >= 0 && s < p.src.num_blocks && d >= 0 && d < p.dst.num_blocks; };
    for (int i = gtid; i < p.num_pages; i += kStep) {
        const int s = p.src_pages[i], d = p.dst_pages[i];
        if (good(s, d)) {
            p.claim[d] = -1;
            if (p.one_pool)
                p.claim[s] = -1;
        }
    }
    cluster_sync();
    for (int i = gtid; i < p.num_pages; i += kStep) {
        const int s = p.src_pages[i], d = p.dst_pages[i];
        if (good(s, d))
            atomicMax(&p.claim[d], i);
    }
}

// ---- the moving kernel ---------------------------------------------------------------------------

struct MoveParams {
    PagePool dst, src;
    const int4 *copies;        // fork, compact: the planned copies, null in copies of listed pages
    const int32_t *num_copies;
    // copies of listed pages
    const int32_t *src_pages;
    const int32_t *dst_pages;
    int32_t num_pages;
    const int32_t *claim;
    bool one_pool;
    // compact: the block table through the page map
    const int32_t *page_map;
    const int32_t *table;
    int64_t table_stride;
    const int32_t *lens;
    int32_t rows;
    int32_t max_blocks;
    int32_t *table_out;
    int64_t table_out_stride;
    unsigned *status;
};

// kGroup threads to a page, kCopyThreads / kGroup pages at a time to a CTA: as few as hold a page in one round of kCopyUnroll
// pieces each, so that a CTA has some 25 KB in flight whatever the size of a page (8000 pages of 6400 bytes in four layers: 5.7
// TB/s, with a whole CTA to a page 3.5).  Two to three CTAs a multiprocessor are level; more disturb DRAM.
template <int kGroup>
__global__ void __launch_bounds__(kCopyThreads) move_pages_kernel(const MoveParams p)
{
    griddep_wait();
    const int tid = threadIdx.x;
    if (p.rows > 0) {
        const int width = max(p.max_blocks, 1);   // (a row without cells has a length to look at)
        const int64_t cells = (int64_t)p.rows * width;
        for (int64_t i = (int64_t)blockIdx.x * kCopyThreads + tid; i < cells; i += (int64_t)gridDim.x * kCopyThreads) {
            const int r = (int)(i / width), j = (int)(i % width);
            const int len = p.lens[r];
            if (j == 0 && len > (int64_t)p.max_blocks * p.dst.page)
                atomicOr(p.status, kStatusBadIndex);
            if (j >= p.max_blocks)
                continue;
            const int np = pages_of(len, p.dst.page, p.max_blocks);
            int v = -1;
            if (j < np) {
                v = p.table[(int64_t)r * p.table_stride + j];
                v = v >= 0 && v < p.dst.num_blocks ? p.page_map[v] : -1;
                if (v < 0)
                    atomicOr(p.status, kStatusBadIndex);
            }
            p.table_out[(int64_t)r * p.table_out_stride + j] = v;
        }
    }
    const int n = p.copies != nullptr ? *p.num_copies : p.num_pages;
    constexpr int kGroups = kCopyThreads / kGroup;
    const int gid = tid % kGroup;
    // a few listed pages are checked against each other here, a pair to a thread, without a plan
    const bool check = kGroups == 1 && p.copies == nullptr && p.claim == nullptr;
    int2 pair = make_int2(-1, -1);
    if (check && tid < n)
        pair = make_int2(p.src_pages[tid], p.dst_pages[tid]);
    const bool pair_good = pair.x >= 0 && pair.x < p.src.num_blocks && pair.y >= 0 && pair.y < p.dst.num_blocks;
    const int64_t units = (int64_t)n * p.dst.num_layers;
    const int64_t page_bytes = (int64_t)p.dst.page * p.dst.entry_bytes;
    for (int64_t u = (int64_t)blockIdx.x * kGroups + tid / kGroup; u < units; u += (int64_t)gridDim.x * kGroups) {
        const int i = (int)(u / p.dst.num_layers), layer = (int)(u % p.dst.num_layers);
        int4 c;
        if (p.copies != nullptr) {
            c = p.copies[i];
        } else {
            c = make_int4(p.src_pages[i], p.dst_pages[i], p.dst.page, 0);
            const bool good = c.x >= 0 && c.x < p.src.num_blocks && c.y >= 0 && c.y < p.dst.num_blocks;
            bool later, target;   // a later pair has this target; the source is a target of the call
            if (check) {
                later = __syncthreads_or(pair_good && tid > i && pair.y == c.y);
                target = __syncthreads_or(pair_good && p.one_pool && pair.y == c.x);
            } else {
                later = good && p.claim[c.y] != i;
                target = good && p.one_pool && p.claim[c.x] != -1;
            }
            if (!good || later || target) {
                if ((!good || (target && !later)) && gid == 0 && layer == 0)
                    atomicOr(p.status, kStatusBadIndex);
                continue;
            }
        }
        const uint4 *s = reinterpret_cast<const uint4 *>(p.src.base + layer * p.src.layer_stride + c.x * page_bytes);
        uint4 *d = reinterpret_cast<uint4 *>(p.dst.base + layer * p.dst.layer_stride + c.y * page_bytes);
        const int pieces = (int)((int64_t)c.z * p.dst.entry_bytes / 16);
        for (int i0 = 0; i0 < pieces; i0 += kCopyUnroll * kGroup) {
            uint4 v[kCopyUnroll];
#pragma unroll
            for (int k = 0; k < kCopyUnroll; ++k)
                if (i0 + k * kGroup + gid < pieces)
                    v[k] = __ldcs(s + i0 + k * kGroup + gid);
#pragma unroll
            for (int k = 0; k < kCopyUnroll; ++k)
                if (i0 + k * kGroup + gid < pieces)
                    __stcs(d + i0 + k * kGroup + gid, v[k]);
        }
    }
}

cudaError_t launch_move(const MoveParams &m, int sms, cudaStream_t stream)
{
    const int64_t pieces = (int64_t)m.dst.page * m.dst.entry_bytes / 16;
    const bool check = m.copies == nullptr && m.claim == nullptr;   // (by whole CTAs)
    const auto kernel = check || pieces > kCopyUnroll * 128 ? move_pages_kernel<256>
                        : pieces > kCopyUnroll * 64         ? move_pages_kernel<128>
                                                            : move_pages_kernel<64>;
    return launch_dependent(kernel, dim3((unsigned)(sms * 3)), kCopyThreads, 0, stream, m);
}

}  // namespace

cudaError_t launch_fork(const ForkParams &p, int sms, cudaStream_t stream)
{
    cudaError_t e;
    if (p.pool.num_blocks <= kSmallPages && p.rows <= kSmallRows && p.rows_out <= kSmallRows &&
        (int64_t)std::max(p.rows, p.rows_out) * p.max_blocks <= kSmallCells) {
        const int bytes = 4 * (3 * p.pool.num_blocks + 5 * p.rows + 2 * p.rows_out);
        e = set_smem_once(reinterpret_cast<const void *>(fork_plan_small_kernel), bytes, kAttrForkSmall);
        if (e != cudaSuccess)
            return e;
        e = launch_dependent(fork_plan_small_kernel, dim3(1), kPlanThreads, (size_t)bytes, stream, p);
    } else {
        e = launch_dependent(fork_plan_kernel, dim3(kCluster), kPlanThreads, 0, stream, p);
    }
    if (e != cudaSuccess)
        return e;
    MoveParams m{};
    m.dst = m.src = p.pool;
    m.copies = p.copies;
    m.num_copies = p.num_copies;
    return launch_move(m, sms, stream);
}

cudaError_t launch_compact(const CompactParams &p, int sms, cudaStream_t stream)
{
    cudaError_t e;
    if (p.pool.num_blocks <= kSmallPages) {
        const int bytes = 12 * p.pool.num_blocks + 8;
        e = set_smem_once(reinterpret_cast<const void *>(compact_plan_small_kernel), bytes, kAttrCompactSmall);
        if (e != cudaSuccess)
            return e;
        e = launch_dependent(compact_plan_small_kernel, dim3(1), kPlanThreads, (size_t)bytes, stream, p);
    } else {
        e = launch_dependent(compact_plan_kernel, dim3(kCluster), kPlanThreads, 0, stream, p);
    }
    if (e != cudaSuccess)
        return e;
    MoveParams m{};
    m.dst = m.src = p.pool;
    m.copies = p.copies;
    m.num_copies = p.num_copies;
    m.page_map = p.page_map;
    m.table = p.table;
    m.table_stride = p.table_stride;
    m.lens = p.lens;
    m.rows = p.rows;
    m.max_blocks = p.max_blocks;
    m.table_out = p.table_out;
    m.table_out_stride = p.table_out_stride;
    m.status = p.status;
    return launch_move(m, sms, stream);
}

cudaError_t launch_copy_pages(const CopyPagesParams &p, int sms, cudaStream_t stream)
{
    // A short list goes without a plan (8 pages of 25600 bytes in 1, 8 and 40 layers: 2.1, 2.2 and 3.4 us, with it 4.0, 4.1 and
    // 5.3; 256 pages: 3.4, 13.9 and 84 against 5.7, 17.9 and 91).  Pages that would not take a whole CTA then do, with two
    // barriers each: up to about 2048 of them, over all layers, that still costs less than the plan (6400 bytes, 256 pages in 8
    // layers: 5.5 against 6.8, in 40: 33 against 21; 400 bytes: 5.2 against 5.0, and 18.7 against 8.5).
    const int64_t pieces = (int64_t)p.dst.page * p.dst.entry_bytes / 16;
    const bool few = p.num_pages <= kCopyThreads &&
                     (pieces > kCopyUnroll * 128 || (int64_t)p.num_pages * p.dst.num_layers <= kFewSmall);
    if (!few) {
        const cudaError_t e = launch_dependent(copy_plan_kernel, dim3(kCluster), kPlanThreads, 0, stream, p);
        if (e != cudaSuccess)
            return e;
    }
    MoveParams m{};
    m.dst = p.dst;
    m.src = p.src;
    m.src_pages = p.src_pages;
    m.dst_pages = p.dst_pages;
    m.num_pages = p.num_pages;
    m.claim = few ? nullptr : p.claim;
    m.one_pool = p.one_pool;
    m.status = p.status;
    return launch_move(m, sms, stream);
}

}  // namespace dsv4
