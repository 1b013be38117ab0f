// evict.cu -- eviction from a paged cache by accumulated attention weight.
//
// A row of n > limit entries keeps its first `first`, its last `recent` and, of those between, the heaviest
// (budget in all), in their order.  Entry i of the new row is entry kept(i) >= i of the old one, so everything moves down:
//   kept(i) = i                             i < first
//             first + picked[i - first]     the picked ones
//             n - budget + i                the recent ones
// Three launches: the selection, a plan (pages, lengths, counts), and the moves; two for a few short rows, whose selection and plan
// are one cluster's (4 rows of 300 to 700: 15.7 us with three, 13.8 with two).
//
// The selection.  Rows of up to 4096 entries between the first and the recent ones: a CTA a row, an entry's weight as an
// order-preserving 32-bit key in a register.  The lightest kept key is found two bits at a time by counting (no histograms,
// whose atomics meet at the many entries of weight 0), from what is known of weights: whether it is 0 is asked first, and the
// search ends at a threshold that exactly the wanted number of keys reaches.  Longer rows go through the radix select of
// topk.cu, with a launch ahead of it that counts the entries.  In us, counting against that: 4 rows of 700 7 / 15, 32 of 2500 10 /
// 14, 64 of 12000 30 / 19 (two CTAs a row), one of 131000 36 / 25 (eight).
//
// The plan.  A page of the new row whose entries all stay where they are and that is full stays, shared or not.  The other
// pages are written: in place where the row alone holds the page, into a free page (lowest first) otherwise.  Pages past
// the new end, and those replaced by a free one, lose a reference.  One cluster, a thread a cell.
//
// The moves go through every layer, in place and in one pass over the bytes.  A row's new entries are cut into tiles; a
// CTA reads the sources of a tile into registers, says so in a bitmap, waits until the tiles before it whose sources its own
// writes would overwrite have been read (sources lie at or past their targets, so only earlier tiles can be in the way),
// and writes.  Tiles are handed out by a ticket in that order, and a CTA draws its next one while it has one in hand, so a
// tile may wait for one that nobody has begun.  All the same every wait ends: a CTA says that its tile has been read before it
// waits, so the lowest ticket that has not been read is either being read, or it is the next one of a CTA whose tile in hand,
// a lower ticket, waits for still lower ones, which have all been read.  Each wait is bounded besides.  The weights go the
// same way, in tiles of their own.
#include <algorithm>
#include <climits>

#include "serving.h"

namespace dsv4 {
namespace {

constexpr int kCluster = 8;
constexpr int kPlanThreads = 1024;
constexpr int kFewRows = 8, kFewCells = 8192, kFewPages = 32768;   // what one CTA plans
constexpr int kMoveThreads = 256;
constexpr int kUnroll = 8;                                  // 16-byte pieces a thread holds
constexpr int kTileBytes = 16 * kMoveThreads * kUnroll;     // 32 KB
constexpr int kMaxTile = 512;                               // entries
constexpr int kWeightTile = kMoveThreads * kUnroll;         // weights
constexpr int kZeroTile = 4 * kWeightTile;
constexpr int kSelectThreads = 1024;
constexpr int kSelectEach = 4;                              // keys of a thread
constexpr int kWide = 1 << 30;                              // positions and tiles' ends of rows up to this fit 32 bits with room
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

// Larger weight -> larger key; -0 and +0 share a key; NaN below every number.
__device__ __forceinline__ uint32_t order_key(float x)
{
    const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
    return x != x ? 0u : u & 0x80000000u ? ~u : u | 0x80000000u;
}

// The heaviest entries of a row between its first and its recent ones, of up to kEach * kSelectThreads (key u of thread t: entry
// u * kSelectThreads + t), and the lowest that is not among them.
template <int kEach>
__device__ __forceinline__ void select_row(const EvictParams &p, int r)
{
    __shared__ uint2 count[2][32];
    __shared__ int wsum[32];
    __shared__ uint32_t cells[32 * kEach];       // (keys above, keys equal) of each warp's 32 entries, in order; then sums
    __shared__ int lowest;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    bool over;
    const int n = length_of(p, r, &over), k = p.budget - p.first - p.recent;
    if (n <= p.limit)
        return;
    const int len = n - p.first - p.recent;      // > k
    const float *w = p.weights + (int64_t)r * p.weights_stride + p.first;
    uint32_t key[kEach];
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
        const int i = u * kSelectThreads + tid;
        key[u] = i < len ? order_key(__ldcg(w + i)) : 0u;   // (0 where there is no entry: no threshold is that low)
    }
    if (tid == 0)
        lowest = INT_MAX;
    int turn = 0;
    // the threads' sums of (x's halves, y)
    auto sum_all = [&](uint32_t x, uint32_t y) {
        x = __reduce_add_sync(0xffffffffu, x);
        y = __reduce_add_sync(0xffffffffu, y);
        uint2 *slot = count[turn++ & 1];         // (two places in turn: one barrier a round)
        if (lane == 0)
            slot[warp] = make_uint2(x, y);
        __syncthreads();
        x = __reduce_add_sync(0xffffffffu, slot[lane].x);
        return make_int3((int)(x & 0xFFFFu), (int)(x >> 16), (int)__reduce_add_sync(0xffffffffu, slot[lane].y));
    };
    // ---- the k-th largest key `top`, and how many keys are larger
    constexpr uint32_t kZero = 0x80000000u;      // of a weight of 0
    uint32_t top = 0u;
    int more;
    {
        uint32_t c = 0u;
#pragma unroll
        for (int u = 0; u < kEach; ++u)
            c += (key[u] > kZero ? 1u : 0u) + (key[u] >= kZero ? 0x10000u : 0u);
        const int3 s = sum_all(c, 0u);
        const int gt = s.x, ge = s.y;
        bool done = false;
        if (ge >= k) {
            top = kZero;
            more = gt;
            done = gt < k;
        } else {
            more = ge;
        }
#pragma unroll 1
        for (int s0 = 29; !done; s0 -= 2) {      // bits s0 + 1 and s0 (the last round: bit 0 alone)
            const uint32_t step = s0 >= 0 ? 1u << s0 : 1u;
            const uint32_t t1 = top + step, t2 = s0 >= 0 ? t1 + step : ~0u, t3 = s0 >= 0 ? t2 + step : ~0u;
            uint32_t x = 0u, y = 0u;
#pragma unroll
            for (int u = 0; u < kEach; ++u) {
                x += (key[u] >= t1 ? 1u : 0u) + (key[u] >= t2 ? 0x10000u : 0u);
                y += key[u] >= t3 ? 1u : 0u;
            }
            const int3 sum = sum_all(x, y);
            const int c1 = sum.x, c2 = sum.y, c3 = sum.z;
            const bool one = s0 < 0;
            uint32_t next = top;
            int c = -1;                          // keys that reach `next`
            if (!one && c3 >= k) {
                next = t3;
                c = c3;
            } else if (!one && c2 >= k) {
                next = t2;
                c = c2;
                more = c3;
            } else if (c1 >= k) {
                next = t1;
                c = c1;
                more = one ? more : c2;
            } else {
                more = c1;
            }
            top = next;
            done = one;
            if (c == k) {                        // exactly the keys that reach it
                top = next - 1u;
                more = k;
                done = true;
            }
        }
    }
    const int take = k - more;                   // of the keys equal to top, the first ones
    // ---- where each warp's 32 entries begin in the list
    uint32_t above[kEach], equal[kEach];
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
        const bool in = u * kSelectThreads + tid < len;
        above[u] = __ballot_sync(0xffffffffu, in && key[u] > top);
        equal[u] = __ballot_sync(0xffffffffu, in && key[u] == top);
        if (lane == 0)
            cells[32 * u + warp] = (uint32_t)__popc(above[u]) | ((uint32_t)__popc(equal[u]) << 16);
    }
    __syncthreads();
    int total;
    const uint32_t cell = tid < 32 * kEach ? cells[tid] : 0u;
    const uint32_t before = (uint32_t)cta_scan((int)cell, wsum, &total);   // (each half below 2^15: no carry between them)
    if (tid < 32 * kEach)
        cells[tid] = before;
    __syncthreads();
    int32_t *out = p.picked + (int64_t)r * k;
    int left = INT_MAX;                          // the lowest entry of this thread that is not kept
#pragma unroll
    for (int u = kEach - 1; u >= 0; --u) {
        const int i = u * kSelectThreads + tid;
        const uint32_t at = cells[32 * u + warp], below = (1u << lane) - 1u;
        const int a = (int)(at & 0xFFFFu) + __popc(above[u] & below), e = (int)(at >> 16) + __popc(equal[u] & below);
        const bool kept = ((above[u] >> lane) & 1u) || (((equal[u] >> lane) & 1u) && e < take);
        if (kept)
            out[a + min(e, take)] = i;
        else if (i < len)
            left = i;
    }
    left = __reduce_min_sync(0xffffffffu, left);
    if (lane == 0)
        atomicMin(&lowest, left);
    __syncthreads();
    if (tid == 0)
        p.moved[r] = p.first + lowest;
}

// The plan, by a cluster of kCluster CTAs, or (kFew) by one.
template <bool kFew>
__device__ __forceinline__ void make_plan(const EvictParams &p)
{
    __shared__ int wsum[32];
    __shared__ int count;
    constexpr int kParts = kFew ? 1 : kCluster, kStep = kParts * kPlanThreads, kWarps = kStep / 32;
    const int rank = kFew ? 0 : cluster_rank(), tid = threadIdx.x, lane = tid & 31;
    const int gtid = rank * kPlanThreads + tid, gwarp = gtid >> 5;
    const int B = p.pool.num_blocks, page = p.pool.page;
    auto sync = [&]() {
        if (kFew)
            __syncthreads();
        else
            cluster_sync();
    };

    // ---- each row's new length, and the first entry that is written
    for (int r = gwarp; r < p.rows; r += kWarps) {
        bool over;
        const int n = length_of(p, r, &over);
        const bool cut = n > p.limit;
        const int m = cut ? p.budget : n;
        int f = n;
        if (cut && p.selected) {
            f = min(__ldcg(p.moved + r), m);
        } else if (cut) {   // the lowest i with kept(i) != i (kept(i) - i does not fall), 32 places at a time
            int a = 0, z = m;
            while (a < z) {
                const unsigned step = ((unsigned)(z - a) + 31u) / 32u, i = a + lane * step;   // (rows may have nearly 2^31 entries)
                const unsigned still = __ballot_sync(0xffffffffu, i < (unsigned)z && kept(p, r, n, (int)i) == (int)i);
                const int c = __popc(still);          // (a run of the low lanes)
                z = c == 0 ? a : (int)min((unsigned)z, a + c * step);
                a = c == 0 ? a : (int)(a + (c - 1) * step + 1u);
            }
            f = a;
        }
        __syncwarp();
        if (lane == 0) {
            p.need[r] = 0;
            p.moved[r] = f;
            p.lens_out[r] = m;
            if (over)
                atomicOr(p.status, kStatusBadIndex);
        }
    }
    if (p.refs_out != p.refs)
        for (int i = gtid; i < B; i += kStep)
            p.refs_out[i] = p.refs[i];
    const int64_t words = (int64_t)p.rows * (p.columns * p.words + p.weight_words);
    for (int64_t i = gtid; i < words; i += kStep)
        p.read[i] = 0u;
    if (gtid == 0)
        *p.ticket = 0;
    sync();

    // ---- the cells: pages as they stand, -2 for those to take
    const int64_t cells = (int64_t)p.rows * p.max_blocks;
    for (int64_t x = gtid; x < cells; x += kStep) {
        const int r = (int)((unsigned long long)x / (unsigned)p.max_blocks), j = (int)(x - (int64_t)r * p.max_blocks);
        bool over;
        const int n = length_of(p, r, &over);
        const int m = __ldcg(p.lens_out + r);
        int v = -1;
        if (j < pages_of(n, page)) {
            v = p.table[(int64_t)r * p.table_stride + j];
            if (v < 0 || v >= B) {
                atomicOr(p.status, kStatusBadIndex);
                v = -1;
            }
        }
        if (j >= pages_of(m, page)) {
            v = -1;
        } else if (v >= 0 && m < n && j >= min(__ldcg(p.moved + r), m) / page && p.refs[v] != 1) {
            v = -2;
            atomicAdd(p.need + r, 1);
        }
        p.table_out[(int64_t)r * p.table_out_stride + j] = v;
    }
    sync();

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
    if (wanted > 0) {
        // ---- the free pages' list, lowest first
        const int part = (B + kParts - 1) / kParts;
        const int lo = min(B, rank * part), hi = min(B, lo + part);
        int mine = 0, before = 0, num_free = 0;
        for (int i = lo + tid; i < hi; i += kPlanThreads)
            mine += p.refs[i] == 0;
        cta_scan(mine, wsum, &total);
        if (tid == 0)
            count = total;
        sync();
        for (int k = 0; k < kParts; ++k) {
            const int v = kFew ? count : ld_rank(&count, k);
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
        sync();

        // ---- the new pages into the rows that take some
        for (int r = gwarp; r < p.rows; r += kWarps) {
            const int need = __ldcg(p.need + r), off = __ldcg(p.offset + r);
            if (need == 0)
                continue;
            bool over;
            const int n = length_of(p, r, &over);
            const int32_t *src = p.table + (int64_t)r * p.table_stride;
            int32_t *dst = p.table_out + (int64_t)r * p.table_out_stride;
            if (need > num_free - off) {   // not enough pages: the row stays as it was
                for (int j = lane; j < pages_of(n, page); j += 32) {
                    const int v = src[j];
                    dst[j] = v >= 0 && v < B ? v : -1;
                }
                if (lane == 0) {
                    p.moved[r] = n;
                    p.lens_out[r] = n;
                    atomicOr(p.status, kStatusBadIndex);
                }
                continue;
            }
            const int np = pages_of(p.budget, page);
            int at = off;
            for (int j0 = 0; j0 < np; j0 += 32) {
                const int j = j0 + lane;
                const bool take = j < np && __ldcg(dst + j) == -2;
                const unsigned m = __ballot_sync(0xffffffffu, take);
                if (take) {
                    const int q = __ldcg(p.free_list + at + __popc(m & ((1u << lane) - 1u)));
                    dst[j] = q;
                    p.refs_out[q] = 1;
                    atomicSub(&p.refs_out[src[j]], 1);
                }
                at += __popc(m);
            }
        }
        sync();   // (rows that stay as they were have their length again)
    }

    // ---- the pages past the new ends lose a reference
    for (int64_t x = gtid; x < cells; x += kStep) {
        const int r = (int)((unsigned long long)x / (unsigned)p.max_blocks), j = (int)(x - (int64_t)r * p.max_blocks);
        bool over;
        const int n = length_of(p, r, &over), m = __ldcg(p.lens_out + r);
        if (m < n && j >= pages_of(m, page) && j < pages_of(n, page)) {
            const int v = p.table[(int64_t)r * p.table_stride + j];
            if (v >= 0 && v < B)
                atomicSub(&p.refs_out[v], 1);
        }
    }
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kPlanThreads) evict_plan_kernel(const EvictParams p)
{
    griddep_wait();
    griddep_launch();   // (the moving kernel waits for this grid itself)
    make_plan<false>(p);
}

template <int kEach>
__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const EvictParams p)
{
    griddep_wait();
    griddep_launch();
    select_row<kEach>(p, blockIdx.x);
}

// Selection and plan of a cluster's rows, a CTA each.
template <int kEach>
__global__ void __launch_bounds__(kSelectThreads) evict_few_kernel(const EvictParams p)
{
    griddep_wait();
    griddep_launch();
    select_row<kEach>(p, blockIdx.x);
    cluster_sync();
    if (blockIdx.x == 0)
        make_plan<true>(p);
}

// Waits until the tiles [first, tile) of a bitmap have been read, by a warp; false if that took too long.
__device__ __forceinline__ bool wait_read(const uint32_t *bits, int first, int tile, int lane)
{
    bool lost = false;
    for (int w = first / 32 + lane; first < tile && w <= (tile - 1) / 32; w += 32) {
        uint32_t want = 0xffffffffu;
        if (w == first / 32)
            want &= 0xffffffffu << (first & 31);
        if (w == tile / 32)
            want &= (1u << (tile & 31)) - 1u;
        const long long t0 = clock64();
        while ((*reinterpret_cast<const volatile uint32_t *>(bits + w) & want) != want)
            if (clock64() - t0 > kWaitCycles) {
                lost = true;
                break;
            }
    }
    __threadfence();
    return !lost;
}

// In the order of the tickets: the rows' weights in tiles (of all rows the first, then the second, ..), what has to be zero after
// them, then the entries' tiles (of all rows and columns the first, then the second, ..).
// Index: int, or int64_t where rows or weights past kWide would wrap around (with it for all, a row of 131000 took 1 % longer).
template <typename Index>
__global__ void __launch_bounds__(kMoveThreads, 4) evict_move_kernel(const EvictParams p)
{
    __shared__ int64_t src_at[kMaxTile], dst_at[kMaxTile];   // byte offsets in the layer; -1: not written
    __shared__ int next;
    const int tid = threadIdx.x;
    const int page = p.pool.page, entry = p.pool.entry_bytes;
    const int per_tile = p.rows * p.columns;
    const int weight_tickets = p.rows * p.weight_tiles, zero_tickets = p.rows * p.zero_tiles;
    const int64_t tickets = (int64_t)weight_tickets + zero_tickets + (int64_t)per_tile * p.tiles;
    const int entry_columns = (entry + p.column_bytes - 1) / p.column_bytes;
    const bool same_weights = p.weights == p.weights_out;
    griddep_wait();
    if (tid == 0)
        next = atomicAdd(p.ticket, 1);
    while (true) {
        __syncthreads();
        const int ticket = next;
        if (ticket >= tickets)
            return;
        __syncthreads();   // (`next` has been read; src_at and dst_at are free)
        if (tid == 0)      // (the next one is on its way meanwhile; one and no more, or waits might not end)
            next = atomicAdd(p.ticket, 1);
        if (ticket < weight_tickets + zero_tickets) {
            const bool zeros = ticket >= weight_tickets;
            const int x = zeros ? ticket - weight_tickets : ticket, r = x % p.rows, tile = x / p.rows;
            bool over;
            const int n = length_of(p, r, &over), m = __ldcg(p.lens_out + r);
            const float *src = p.weights + (int64_t)r * p.weights_stride;
            float *dst = p.weights_out + (int64_t)r * p.weights_out_stride;
            uint32_t *bits = p.read + (int64_t)p.rows * p.columns * p.words + (int64_t)r * p.weight_words;
            if (zeros) {   // [m, width), once every source has been read
                const Index i0 = tile * kZeroTile, i1 = min((Index)p.weights_width, i0 + kZeroTile);
                bool lost = false;
                if (i1 <= m)
                    continue;
                if (same_weights && m < n && i0 < n && tid < 32)
                    lost = !wait_read(bits, __ldcg(p.moved + r) / kWeightTile, (m - 1) / kWeightTile + 1, tid);
                if (__syncthreads_or(lost)) {
                    if (tid == 0)
                        atomicOr(p.status, kStatusTimeout);
                    continue;
                }
                for (Index i = max((Index)m, i0) + tid; i < i1; i += kMoveThreads)
                    dst[i] = 0.f;
                continue;
            }
            const int i0 = tile * kWeightTile, f = m < n ? __ldcg(p.moved + r) : n;
            // (a row that is not cut may be longer than a tile for each of the budget's entries)
            for (Index j0 = i0; j0 < m; j0 += (Index)p.weight_tiles * kWeightTile) {
                if (same_weights && j0 + kWeightTile <= f)
                    continue;   // (nothing moves)
                float v[kUnroll];
                float sum = 0.f;
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    const Index i = j0 + u * kMoveThreads + tid;
                    v[u] = i < m ? __ldcg(src + (i < f ? i : (Index)kept(p, r, n, (int)i))) : 0.f;
                    sum = fmaxf(sum, v[u]);
                }
                bool lost = false;
                __syncthreads_or(sum > 0.f);   // (takes a value that depends on every load, so that they have all returned)
                if (same_weights && m < n) {
                    if (tid == 0) {
                        __threadfence();
                        atomicOr(bits + tile / 32, 1u << (tile & 31));
                    }
                    if (tid < 32)
                        lost = !wait_read(bits, min(tile, max(f, (int)j0 - (n - m)) / kWeightTile), tile, tid);
                }
                if (__syncthreads_or(lost)) {
                    if (tid == 0)
                        atomicOr(p.status, kStatusTimeout);
                    continue;
                }
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    const Index i = j0 + u * kMoveThreads + tid;
                    if (i < m)
                        dst[i] = v[u];
                }
            }
            continue;
        }
        const int tile = (ticket - weight_tickets - zero_tickets) / per_tile;
        const int unit = (ticket - weight_tickets - zero_tickets) - tile * per_tile;
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
        const bool lost = tid < 32 && !wait_read(bits, first, tile, tid);
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

EvictShape evict_shape(int num_layers, int entry_bytes, int budget, int weights_width)
{
    EvictShape s;
    s.column_bytes = std::min(entry_bytes, kTileBytes);
    s.tile = std::min(kMaxTile, kTileBytes / s.column_bytes);
    s.columns = num_layers * ((entry_bytes + s.column_bytes - 1) / s.column_bytes);
    s.tiles = (budget - 1) / s.tile + 1;
    s.words = (s.tiles + 31) / 32;
    s.weight_tiles = (budget - 1) / kWeightTile + 1;
    s.weight_words = (s.weight_tiles + 31) / 32;
    s.zero_tiles = weights_width / kZeroTile + 1;
    return s;
}

cudaError_t launch_evict(EvictParams p, int sms, cudaStream_t stream)
{
    const int picked = p.budget - p.first - p.recent;
    const int64_t most = (int64_t)p.max_blocks * p.pool.page;    // of a row's entries
    // four moving CTAs to a multiprocessor, or as many as there are tiles
    const int64_t tickets = (int64_t)p.rows * (p.weight_tiles + p.zero_tiles + (int64_t)p.columns * p.tiles);
    const auto move = std::max<int64_t>(most, p.weights_width) > kWide ? evict_move_kernel<int64_t> : evict_move_kernel<int>;
    const dim3 movers((unsigned)std::max<int64_t>(1, std::min<int64_t>(4ll * sms, tickets)));
    if (picked > 0 && p.rows > 0 && most > p.limit) {
        const int width = (int)(most - p.first - p.recent);
        cudaError_t e;
        if (width <= kSelectThreads * kSelectEach) {
            p.selected = true;
            if (p.rows <= kFewRows && (int64_t)p.rows * p.max_blocks <= kFewCells && p.pool.num_blocks <= kFewPages) {
                cudaLaunchConfig_t cfg = {};
                cfg.gridDim = dim3((unsigned)p.rows);
                cfg.blockDim = dim3(kSelectThreads);
                cfg.stream = stream;
                cudaLaunchAttribute attr[2];
                attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
                attr[0].val.programmaticStreamSerializationAllowed = 1;
                attr[1].id = cudaLaunchAttributeClusterDimension;
                attr[1].val.clusterDim.x = (unsigned)p.rows;
                attr[1].val.clusterDim.y = 1;
                attr[1].val.clusterDim.z = 1;
                cfg.attrs = attr;
                cfg.numAttrs = 2;
                e = cudaLaunchKernelEx(&cfg, width <= kSelectThreads ? evict_few_kernel<1> : evict_few_kernel<kSelectEach>, p);
                if (e != cudaSuccess) {
                    (void)cudaGetLastError();
                    return e;
                }
                return launch_dependent(move, movers, kMoveThreads, 0, stream, p);
            }
            e = launch_dependent(width <= kSelectThreads ? evict_select_kernel<1> : evict_select_kernel<kSelectEach>,
                                 dim3((unsigned)p.rows), kSelectThreads, 0, stream, p);
        } else {
            e = launch_dependent(evict_between_kernel, dim3((unsigned)(p.rows + kMoveThreads - 1) / kMoveThreads), kMoveThreads, 0,
                                 stream, p);
            if (e == cudaSuccess)
                e = launch_topk_select(p.weights + p.first, p.weights_stride, width, p.between, p.rows, picked, p.picked, picked,
                                       nullptr, topk_cluster_size(p.rows, width, sms), stream);
            if (e != cudaSuccess)
                (void)cudaGetLastError();
        }
        if (e != cudaSuccess)
            return e;
    }
    const cudaError_t e = launch_dependent(evict_plan_kernel, dim3(kCluster), kPlanThreads, 0, stream, p);
    if (e != cudaSuccess)
        return e;
    return launch_dependent(move, movers, kMoveThreads, 0, stream, p);
}

}  // namespace dsv4
