// evict.cu -- eviction from a paged cache by accumulated attention weight.
//
// A row of n > limit entries keeps its first `first`, its last `recent` and, of those between, the heaviest
// (budget in all), in their order.  Entry i of the new row is entry kept(i) >= i of the old one, so everything moves down:
//   kept(i) = i                             i < first
//             first + picked[i - first]     the picked ones
//             n - budget + i                the recent ones
// The selection (topk.cu: radix select over the weights), a plan (pages, lengths, counts), and the moves.
//
// The plan.  A page of the new row whose entries all stay where they are and that is full stays, shared or not.  The other
// pages are written: in place where the row alone holds the page, into a free page (lowest first) otherwise.  Pages past
// the new end, and those replaced by a free one, lose a reference.
//
// The moves go through every layer, in place and in one pass over the bytes.  A row's new entries are cut into tiles; a
// CTA reads the sources of a tile into registers, says so in a bitmap, waits until the tiles before it whose sources its own
// writes would overwrite have been read (sources lie at or past their targets, so only earlier tiles can be in the way),
// and writes.  Tiles are handed out by a ticket in that order, so those that a tile waits for were begun before it and
// never wait for it; every wait is bounded.
#include <algorithm>
#include <climits>

#include "serving.h"

namespace dsv4 {
namespace {

constexpr int kCluster = 8;
constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kCluster * kPlanThreads / 32;
constexpr int kMoveThreads = 256;
constexpr int kUnroll = 8;                                  // 16-byte pieces a thread holds
constexpr int kTileBytes = 16 * kMoveThreads * kUnroll;     // 32 KB
constexpr int kMaxTile = 512;                               // entries
constexpr long long kWaitCycles = 4000000000LL;             // about two seconds

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
    const int before = __reduce_add_sync(0xffffffffu, lane < warp ? ws : 0);
    *total = __reduce_add_sync(0xffffffffu, ws);
    return before + x - v;
}

__device__ __forceinline__ int pages_of(int len, int page) { return len <= 0 ? 0 : (len - 1) / page + 1; }

// entries that row r holds, as far as the table goes
__device__ __forceinline__ int length_of(const EvictParams &p, int r, bool *cut)
{
    const int len = p.lens[r];
    const int64_t most = (int64_t)p.max_blocks * p.pool.page;
    *cut = len > most;
    return max(0, *cut ? (int)most : len);
}

// the old position of entry i of a row of n entries that is cut
__device__ __forceinline__ int kept(const EvictParams &p, int r, int n, int i)
{
    const int k = p.budget - p.first - p.recent;
    if (i < p.first)
        return i;
    if (i < p.first + k)
        return p.first + __ldcg(p.picked + (int64_t)r * k + (i - p.first));
    return n - p.budget + i;
}

__global__ void __launch_bounds__(kMoveThreads) evict_between_kernel(const EvictParams p)
{
    griddep_wait();
    griddep_launch();
    const int r = blockIdx.x * kMoveThreads + threadIdx.x;
    bool over;
    if (r < p.rows)
        p.between[r] = max(0, length_of(p, r, &over) - p.first - p.recent);
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kPlanThreads) evict_plan_kernel(const EvictParams p)
{
    __shared__ int wsum[32];
    __shared__ int count;
    const int rank = cluster_rank(), tid = threadIdx.x, lane = tid & 31;
    const int gtid = rank * kPlanThreads + tid, gwarp = gtid >> 5;
    constexpr int kStep = kCluster * kPlanThreads;
    const int B = p.pool.num_blocks, page = p.pool.page;
    griddep_wait();
    griddep_launch();   // (the moving kernel waits for this grid itself)

    // ---- each row's pages as they stand, -2 for those to take, and the first entry that is written
    for (int r = gwarp; r < p.rows; r += kPlanWarps) {
        bool over;
        const int n = length_of(p, r, &over);
        const bool cut = n > p.limit;
        const int m = cut ? p.budget : n;
        int f = n;
        if (cut) {   // the lowest i with kept(i) != i (kept(i) - i does not fall), 32 places at a time
            int a = 0, z = m;
            while (a < z) {
                const int step = (z - a + 31) / 32, i = a + lane * step;
                const unsigned still = __ballot_sync(0xffffffffu, i < z && kept(p, r, n, i) == i);
                const int c = __popc(still);          // (a run of the low lanes)
                z = c == 0 ? a : min(z, a + c * step);
                a = c == 0 ? a : a + (c - 1) * step + 1;
            }
            f = a;
        }
        const int stay = cut ? min(f, m) / page : INT_MAX;   // pages that stay
        const int np = pages_of(m, page);
        const int32_t *src = p.table + (int64_t)r * p.table_stride;
        int32_t *dst = p.table_out + (int64_t)r * p.table_out_stride;
        int need = 0;
        for (int j = lane; j < p.max_blocks; j += 32) {
            int v = -1;
            if (j < np) {
                v = src[j];
                if (v < 0 || v >= B) {
                    v = -1;
                } else if (j >= stay && p.refs[v] != 1) {
                    v = -2;
                    ++need;
                }
            }
            dst[j] = v;
        }
        need = __reduce_add_sync(0xffffffffu, need);
        if (lane == 0) {
            p.need[r] = need;
            p.moved[r] = f;
            p.lens_out[r] = m;
            if (over)
                atomicOr(p.status, kStatusBadIndex);
        }
    }
    if (p.refs_out != p.refs)
        for (int i = gtid; i < B; i += kStep)
            p.refs_out[i] = p.refs[i];
    const int64_t words = (int64_t)p.rows * p.columns * p.words;
    for (int64_t i = gtid; i < words; i += kStep)
        p.read[i] = 0u;
    if (gtid == 0)
        *p.ticket = 0;
    cluster_sync();

    // ---- where each row's new pages start in the list of free pages (every CTA the same)
    int wanted = 0, total;
    for (int r0 = 0; r0 < p.rows; r0 += kPlanThreads) {
        const int r = r0 + tid;
        const int n = r < p.rows ? __ldcg(p.need + r) : 0;
        const int before = wanted + cta_scan(n, wsum, &total);
        if (rank == 0 && r < p.rows)
            p.offset[r] = before;
        wanted = min(wanted + total, INT_MAX / 2);
    }
    int num_free = 0;
    if (wanted > 0) {   // the free pages' list, lowest first
        const int part = (B + kCluster - 1) / kCluster;
        const int lo = min(B, rank * part), hi = min(B, lo + part);
        int mine = 0, before = 0;
        for (int i = lo + tid; i < hi; i += kPlanThreads)
            mine += p.refs[i] == 0;
        cta_scan(mine, wsum, &total);
        if (tid == 0)
            count = total;
        cluster_sync();
        for (int k = 0; k < kCluster; ++k) {
            const int v = ld_rank(&count, k);
            before += k < rank ? v : 0;
            num_free += v;
        }
        for (int i0 = lo; i0 < hi && before < wanted; i0 += kPlanThreads) {
            const int i = i0 + tid;
            const bool free = i < hi && p.refs[i] == 0;
            const int at = before + cta_scan(free, wsum, &total);
            if (free && at < wanted)
                p.free_list[at] = i;
            before += total;
        }
    }
    cluster_sync();

    // ---- the new pages into the rows; references
    for (int r = gwarp; r < p.rows; r += kPlanWarps) {
        bool over;
        const int n = length_of(p, r, &over);
        const int need = __ldcg(p.need + r), off = __ldcg(p.offset + r);
        const int32_t *src = p.table + (int64_t)r * p.table_stride;
        int32_t *dst = p.table_out + (int64_t)r * p.table_out_stride;
        const int np_old = pages_of(n, page);
        const bool cut = n > p.limit;
        if (cut && need > 0 && need > num_free - off) {   // not enough pages: the row stays as it was
            for (int j = lane; j < np_old; j += 32) {
                const int v = src[j];
                dst[j] = v >= 0 && v < B ? v : -1;
            }
            if (lane == 0) {
                p.moved[r] = n;
                p.lens_out[r] = n;
                atomicOr(p.status, kStatusBadIndex);
            }
        } else if (cut) {
            const int np = pages_of(p.budget, page);
            int at = off;
            for (int j0 = 0; j0 < np_old; j0 += 32) {
                const int j = j0 + lane;
                const bool take = j < np && dst[j] == -2;
                const unsigned m = __ballot_sync(0xffffffffu, take);
                if (take) {
                    const int q = __ldcg(p.free_list + at + __popc(m & ((1u << lane) - 1u)));
                    dst[j] = q;
                    p.refs_out[q] = 1;
                }
                at += __popc(m);
                const int v = j < np_old ? src[j] : -1;
                if (v >= 0 && v < B && (take || j >= np))
                    atomicSub(&p.refs_out[v], 1);
            }
        }
        for (int j = lane; j < np_old; j += 32)
            if (src[j] < 0 || src[j] >= B)
                atomicOr(p.status, kStatusBadIndex);
    }
}

// Rows' weights (the first tickets, a row each), then the tiles: of all rows and columns the first, then the second, ..
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams p)
{
    __shared__ int64_t src_at[kMaxTile], dst_at[kMaxTile];   // byte offsets in the layer; -1: not written
    __shared__ int next;
    const int tid = threadIdx.x;
    const int page = p.pool.page, entry = p.pool.entry_bytes;
    const int64_t per_tile = (int64_t)p.rows * p.columns;
    const int64_t tickets = p.rows + per_tile * p.tiles;
    const int entry_columns = (entry + p.column_bytes - 1) / p.column_bytes;
    griddep_wait();
    while (true) {
        __syncthreads();   // (`next`, src_at and dst_at are free)
        if (tid == 0)
            next = atomicAdd(p.ticket, 1);
        __syncthreads();
        const int64_t ticket = next;
        if (ticket >= tickets)
            return;
        if (ticket < p.rows) {   // ---- a row's weights
            const int r = (int)ticket;
            bool over;
            const int n = length_of(p, r, &over), m = __ldcg(p.lens_out + r);
            const float *src = p.weights + (int64_t)r * p.weights_stride;
            float *dst = p.weights_out + (int64_t)r * p.weights_out_stride;
            const int f = m < n ? __ldcg(p.moved + r) : n;
            for (int i0 = 0; i0 < m; i0 += kUnroll * kMoveThreads) {
                float v[kUnroll];
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    const int i = i0 + u * kMoveThreads + tid;
                    v[u] = i < m ? __ldcg(src + (i < f ? i : kept(p, r, n, i))) : 0.f;
                }
                __syncthreads();   // (in place: sources lie at or past their targets)
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    const int i = i0 + u * kMoveThreads + tid;
                    if (i < m)
                        dst[i] = v[u];
                }
            }
            __syncthreads();
            for (int i = m + tid; i < p.weights_width; i += kMoveThreads)
                dst[i] = 0.f;
            continue;
        }
        const int tile = (int)((ticket - p.rows) / per_tile);
        const int unit = (int)((ticket - p.rows) % per_tile);
        const int r = unit / p.columns, column = unit % p.columns;
        bool over;
        const int n = length_of(p, r, &over), m = __ldcg(p.lens_out + r), f = __ldcg(p.moved + r);
        const int i0 = tile * p.tile, count = min(p.tile, m - i0);
        // entries before `lo` stay where they are (those of a taken page are all written)
        const int lo = f / page * page;
        if (m == n || count <= 0 || i0 + count <= lo)
            continue;
        const int32_t *old_row = p.table + (int64_t)r * p.table_stride, *new_row = p.table_out + (int64_t)r * p.table_out_stride;
        for (int e = tid; e < count; e += kMoveThreads) {
            const int i = i0 + e;
            int64_t s = -1, d = -1;
            if (i >= lo) {
                const int k = kept(p, r, n, i);
                const int b = __ldcg(old_row + k / page), c = __ldcg(new_row + i / page);
                if (b >= 0 && b < p.pool.num_blocks && c >= 0) {
                    s = ((int64_t)b * page + k % page) * entry;
                    d = ((int64_t)c * page + i % page) * entry;
                }
            }
            src_at[e] = s;
            dst_at[e] = s == d ? -1 : d;
        }
        __syncthreads();
        uint8_t *layer = p.pool.base + (column / entry_columns) * p.pool.layer_stride + (int64_t)(column % entry_columns) * p.column_bytes;
        const int pieces = min(p.column_bytes, entry - (column % entry_columns) * p.column_bytes) / 16;   // per entry
        uint4 v[kUnroll];
        uint32_t any = 0u;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = u * kMoveThreads + tid, e = i / pieces;
            v[u] = make_uint4(0u, 0u, 0u, 0u);
            if (e < count && dst_at[e] >= 0)
                v[u] = __ldcg(reinterpret_cast<const uint4 *>(layer + src_at[e]) + (i - e * pieces));
        }
        // (the barrier takes a value that depends on every load, so that they have all returned)
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            any |= v[u].x ^ v[u].w;
        uint32_t *bits = p.read + ((int64_t)r * p.columns + column) * p.words;
        __syncthreads_or(any != 0u);
        if (tid == 0) {
            __threadfence();
            atomicOr(bits + tile / 32, 1u << (tile & 31));
        }
        // ---- the tiles before this one that may read what it writes: kept(i) - i <= n - m
        const int first = max(lo, i0 - (n - m)) / p.tile;
        bool lost = false;
        if (tid < 32) {
            for (int w = first / 32 + tid; w <= (tile - 1) / 32 && first < tile; w += 32) {
                uint32_t want = 0xffffffffu;
                if (w == first / 32)
                    want &= 0xffffffffu << (first & 31);
                if (w == tile / 32)
                    want &= (1u << (tile & 31)) - 1u;
                const long long t0 = clock64();
                while ((*reinterpret_cast<volatile uint32_t *>(bits + w) & want) != want)
                    if (clock64() - t0 > kWaitCycles) {
                        lost = true;
                        break;
                    }
            }
            __threadfence();
        }
        if (__syncthreads_or(lost)) {   // (never, unless a tile before this one was lost)
            if (tid == 0)
                atomicOr(p.status, kStatusTimeout);
            continue;
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = u * kMoveThreads + tid, e = i / pieces;
            if (e < count && dst_at[e] >= 0)
                __stcg(reinterpret_cast<uint4 *>(layer + dst_at[e]) + (i - e * pieces), v[u]);
        }
    }
}

}  // namespace

EvictShape evict_shape(int num_layers, int entry_bytes, int budget)
{
    EvictShape s;
    s.column_bytes = std::min(entry_bytes, kTileBytes);
    s.tile = std::min(kMaxTile, kTileBytes / s.column_bytes);
    s.columns = num_layers * ((entry_bytes + s.column_bytes - 1) / s.column_bytes);
    s.tiles = (budget - 1) / s.tile + 1;
    s.words = (s.tiles + 31) / 32;
    return s;
}

cudaError_t launch_evict(const EvictParams &p, int sms, cudaStream_t stream)
{
    const int picked = p.budget - p.first - p.recent;
    const int64_t most = (int64_t)p.max_blocks * p.pool.page;    // of a row's entries
    if (picked > 0 && p.rows > 0 && most > p.limit) {
        const int width = (int)(most - p.first - p.recent);
        cudaError_t e = launch_dependent(evict_between_kernel, dim3((unsigned)(p.rows + kMoveThreads - 1) / kMoveThreads),
                                         kMoveThreads, 0, stream, p);
        if (e != cudaSuccess)
            return e;
        e = launch_topk_select(p.weights + p.first, p.weights_stride, width, p.between, p.rows, picked, p.picked, picked, nullptr,
                               topk_cluster_size(p.rows, width, sms), stream);
        if (e != cudaSuccess) {
            (void)cudaGetLastError();
            return e;
        }
    }
    const cudaError_t e = launch_dependent(evict_plan_kernel, dim3(kCluster), kPlanThreads, 0, stream, p);
    if (e != cudaSuccess)
        return e;
    return launch_dependent(evict_move_kernel, dim3((unsigned)(sms * 4)), kMoveThreads, 0, stream, p);
}

}  // namespace dsv4
