// verify.cu -- verification of drafted tokens against the target's probabilities, from given random numbers.
//
// Request b has k drafts d_0 .. d_{k-1} and k + 1 rows of target probabilities p_0 .. p_k (the last one for the token
// after all drafts), and k rows of draft probabilities q_j (or none: then q_j is 1 at d_j and 0 elsewhere).
//   accepted  a = the number of leading j with u_j q_j(d_j) < p_j(d_j)
//   weights   w = max(p_a - q_a, 0) when a < k, p_k when all are accepted
//   token     the lowest i with w_0 + .. + w_i > u_k (w_0 + .. + w_{V-1})
// so that the tokens have the target's distribution.  A greedy request accepts while d_j is its row's largest value
// (the lowest index of equal ones) and then takes that of row a.  Without drafts this is plain sampling.
//
// Only row a decides, so a request reads one row of p and at most one of q.  The order of the steps is therefore: every
// CTA of the request finds a (one load of p and q a draft), the request's cluster sums its row's weights tile by tile, the
// CTA whose part holds the wanted sum finds the tile and then the token.
//
// What is decided next to a border has to be right, so sums are pairs of floats (high, low), good to 2^-40 of themselves at
// the worst: a weight is the exact difference of two floats, and Knuth's two-sum says what every addition loses.  In units of
// 2^-48 of the sum: 26 for the roundings of the residuals in the groups of values, and 3 for each of the additions of two
// pairs on the way from a value to the sum: 4 to 32 groups of a lane, 5 for the lanes, up to 32 tiles of a run, 5 and 3 for
// the runs and the CTAs, 14 in the search (wide tiles have few tiles to a run).  With the residuals of all of a lane's 64 to
// 256 values in one float, a likely token in front of a flat tail took 2^-36.  In fp64, whose rate is a sixty-fourth of
// fp32's here, the search alone took a CTA 20 us.
//
// What bounds it.  Large batches: HBM, and the 15 additions and four comparisons that a pair of values takes.  Loads of a
// thread's next 16 values are issued before any is used: with a load, its use and the next load one behind the other, 256
// requests of 151937 took 217 us.  One request: the chain of dependent loads (row numbers, tokens, probabilities, the row,
// the tile again) and the cluster's barrier.
#include <algorithm>
#include <cuda_bf16.h>
#include <limits.h>
#include <math.h>

#include "serving.h"

namespace dsv4 {
namespace {

constexpr int kThreads = 256;        // four CTAs to a multiprocessor
constexpr int kCtasPerSm = 4;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 6;
constexpr int kDeep = 16;            // values that a thread has in flight
constexpr int kMinTile = 256;        // values whose sum is held for the search
constexpr int kMaxTiles = 1024;      // of a CTA
constexpr int kEach = 8;             // values of the tile that a thread looks at

__device__ __forceinline__ float value(float x) { return x; }
__device__ __forceinline__ float value(__nv_bfloat16 x) { return __bfloat162float(x); }

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The cluster's first barrier, in two halves: no CTA writes to another before that one has begun.
__device__ __forceinline__ void cluster_begun() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait_begun() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// v into the place of `local` in the shared memory of the cluster's CTA `rank`
__device__ __forceinline__ void put_remote(void *local, uint32_t rank, unsigned long long v)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(local)), "r"(rank));
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}

struct Sum {   // hi + lo
    float hi, lo;
};

// x into the sum; returns what rounding lost of it, for the low part
__device__ __forceinline__ float add(Sum &s, float x)
{
    const float t = __fadd_rn(s.hi, x);
    const float b = __fsub_rn(t, s.hi);
    const float r = __fadd_rn(__fsub_rn(s.hi, __fsub_rn(t, b)), __fsub_rn(x, b));
    s.hi = t;
    return r;
}

// max(p - q, 0), exactly (q >= 0; NaN has no weight)
__device__ __forceinline__ Sum difference(float p, float q)
{
    const float d = __fsub_rn(p, q), b = __fsub_rn(d, p);
    const float e = __fsub_rn(__fsub_rn(p, __fsub_rn(d, b)), __fadd_rn(q, b));
    return Sum{fmaxf(d, 0.f), d > 0.f ? e : 0.f};   // (the rounded difference has the exact one's sign)
}

__device__ __forceinline__ Sum normal(float x, float y)   // x + y, exactly (|y| <= |x|)
{
    const float hi = __fadd_rn(x, y);
    return Sum{hi, __fsub_rn(y, __fsub_rn(hi, x))};
}

__device__ __forceinline__ Sum plus(const Sum &a, const Sum &b)   // (of positive sums: within 3 * 2^-48)
{
    Sum s = {a.hi, 0.f};
    const float r = add(s, b.hi);
    return normal(s.hi, __fadd_rn(__fadd_rn(a.lo, b.lo), r));
}

__device__ __forceinline__ bool above(const Sum &a, const Sum &b) { return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo); }

__device__ __forceinline__ Sum scaled(const Sum &a, float power) { return Sum{__fmul_rn(a.hi, power), __fmul_rn(a.lo, power)}; }

__device__ __forceinline__ Sum times(const Sum &a, float u)
{
    const float p = __fmul_rn(a.hi, u);
    return normal(p, __fadd_rn(__fmaf_rn(a.hi, u, -p), __fmul_rn(a.lo, u)));
}

__device__ __forceinline__ Sum shfl(const Sum &s, int lane)
{
    return Sum{__shfl_sync(0xffffffffu, s.hi, lane), __shfl_sync(0xffffffffu, s.lo, lane)};
}

// sums over the lanes before this one and with it, of lanes 0 .. width - 1
__device__ __forceinline__ Sum scan32(Sum x, int lane, int width, Sum &before)
{
#pragma unroll
    for (int d = 1; d < 32; d <<= 1)
        if (d < width) {
            const Sum y = {__shfl_up_sync(0xffffffffu, x.hi, d), __shfl_up_sync(0xffffffffu, x.lo, d)};
            if (lane >= d)
                x = plus(y, x);
        }
    before = Sum{__shfl_up_sync(0xffffffffu, x.hi, 1), __shfl_up_sync(0xffffffffu, x.lo, 1)};
    if (lane == 0)
        before = Sum{0.f, 0.f};
    return x;
}

// whether u y < x, exactly
__device__ __forceinline__ bool product_below(float u, float y, float x)
{
    const float r = __fmul_rn(u, y);   // (rounding is monotone: only a product that rounds to x is in doubt, or a subnormal one)
    if (r == x || fabsf(r) < 1e-30f)
        return (double)u * (double)y < (double)x;
    return r < x;
}

// A request's row of weights: p, less the draft's q, or without the drafted token
template <typename T>
struct Row {
    const T *p, *q;
    int point;         // this value has no weight (-1: none)
    // the sum over [t0, t1), by the lanes of a warp
    template <bool kQ>
    __device__ __forceinline__ Sum sum(int t0, int t1, int lane) const
    {
        constexpr int kLoads = kQ ? kDeep / 2 : kDeep, kStep = 32 * kLoads;
        Sum s = {0.f, 0.f};
#pragma unroll 1
        for (int i0 = t0; i0 < t1; i0 += kStep) {
            T x[kLoads], y[kLoads];
            const T *px = p + i0 + lane, *py = q + i0 + lane;
            if (i0 + kStep <= t1 && (unsigned)(point - i0) >= (unsigned)kStep) {   // all of them count
#pragma unroll
                for (int u = 0; u < kLoads; ++u) {
                    x[u] = px[32 * u];
                    if (kQ)
                        y[u] = py[32 * u];
                }
            } else {
#pragma unroll
                for (int u = 0; u < kLoads; ++u) {
                    const int i = i0 + 32 * u + lane;
                    const bool counts = i < t1 && i != point;
                    x[u] = counts ? px[32 * u] : T(0.f);
                    if (kQ)
                        y[u] = counts ? py[32 * u] : T(0.f);
                }
            }
            // a group's sum by halves, its additions' residuals beside it: small against the group, not against the lane's sum
            float v[kLoads], lost = 0.f;
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
                const Sum w = kQ ? difference(value(x[u]), fmaxf(value(y[u]), 0.f)) : Sum{fmaxf(value(x[u]), 0.f), 0.f};
                v[u] = w.hi;
                if (kQ)
                    lost = __fadd_rn(lost, w.lo);
            }
#pragma unroll
            for (int d = 1; d < kLoads; d <<= 1)
#pragma unroll
                for (int u = 0; u < kLoads; u += 2 * d) {
                    Sum pair = {v[u], 0.f};
                    lost = __fadd_rn(lost, add(pair, v[u + d]));
                    v[u] = pair.hi;
                }
            s = plus(s, normal(v[0], lost));
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            const float hi = __shfl_xor_sync(0xffffffffu, s.hi, d), lo = __shfl_xor_sync(0xffffffffu, s.lo, d);
            s = plus(s, Sum{hi, lo});
        }
        return s;
    }
};

template <typename T>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) verify_kernel(const VerifyParams p)
{
    __shared__ Sum tile_sum[kMaxTiles];
    __shared__ Sum totals[kMaxCluster];                       // the cluster's parts of the row
    __shared__ unsigned long long bests[2][kMaxCluster];      // greedy: (order key of the value, ~index)
    __shared__ unsigned long long wbest[kWarps];
    __shared__ Sum wscan[kWarps];
    __shared__ Sum want, start;
    __shared__ float lift;
    __shared__ int owner, chosen, found, last_positive;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = p.cluster, b = blockIdx.x / C;
    const int rank = C > 1 ? (int)cluster_rank() : 0;
    const T *target = static_cast<const T *>(p.target), *draft = static_cast<const T *>(p.draft);
    const int V = p.vocab;
    if (C > 1)
        cluster_begun();
    griddep_wait();
    griddep_launch();

    const int base = p.start[0], row0 = p.start[b] - base, rows = p.start[b + 1] - p.start[b];
    const int d0 = row0 - b, k = rows - 1;   // (every request before this one has a row more than drafts)
    int32_t *out = p.out + (int64_t)b * p.out_stride;
    const bool ok = rows >= 1 && rows <= p.num_rows && row0 >= 0 && row0 <= p.num_rows - rows && d0 >= 0 && d0 <= p.num_drafts - k &&
                    rows <= p.out_width;
    if (!ok) {   // (the same in every CTA of the cluster)
        if (C > 1)
            cluster_wait_begun();
        if (rank == 0) {
            for (int j = tid; j < p.out_width; j += kThreads)
                out[j] = -1;
            if (tid == 0) {
                p.accepted[b] = 0;
                if (p.seq != nullptr)
                    p.seq_out[b] = p.seq[b];
                atomicOr(p.status, kStatusBadIndex);
            }
        }
        return;
    }
    const bool greedy = p.greedy != nullptr && p.greedy[b] != 0;
    // this CTA's part of a row
    const int part = ((V + C - 1) / C + p.tile - 1) / p.tile * p.tile;
    const int lo = min(V, rank * part), hi = min(V, lo + part);

    int a = 0;
    if (greedy) {
        int token;
        if (C > 1)
            cluster_wait_begun();
        for (int j = 0;; ++j) {   // row j: its largest value, the lowest index of equal ones
            const T *row = target + (int64_t)(row0 + j) * p.target_stride;
            float best = -INFINITY;
            int at = INT_MAX;
            for (int i0 = lo + tid; i0 < hi; i0 += kDeep * kThreads) {
                T x[kDeep];
#pragma unroll
                for (int u = 0; u < kDeep; ++u)
                    x[u] = row[min(i0 + u * kThreads, hi - 1)];
#pragma unroll
                for (int u = 0; u < kDeep; ++u) {
                    const int i = i0 + u * kThreads;
                    const float v = value(x[u]);
                    if (i < hi && (v > best || (v == best && at == INT_MAX))) {
                        best = v;
                        at = i;
                    }
                }
            }
            if (best == 0.f)
                best = 0.f;   // (-0 is +0)
            const uint32_t bits = __float_as_uint(best);
            unsigned long long key = at == INT_MAX ? 0ull
                                                   : ((unsigned long long)(bits & 0x80000000u ? ~bits : bits | 0x80000000u) << 32) |
                                                         (uint32_t)~at;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1)
                key = max(key, __shfl_xor_sync(0xffffffffu, key, d));
            if (lane == 0)
                wbest[warp] = key;
            __syncthreads();
            key = wbest[lane % kWarps];
#pragma unroll
            for (int d = kWarps / 2; d > 0; d >>= 1)
                key = max(key, __shfl_xor_sync(0xffffffffu, key, d));
            if (C > 1) {   // (two places in turn: a CTA may be a row ahead of those that still read)
                if (tid < C)
                    put_remote(&bests[j & 1][rank], tid, key);
                cluster_barrier();
                for (int r = 0; r < C; ++r)
                    key = max(key, bests[j & 1][r]);
            }
            token = key == 0ull ? -1 : (int)~(uint32_t)key;
            a = j;
            if (j == k || token < 0 || token != p.tokens[d0 + j])
                break;
            __syncthreads();   // wbest is written again
        }
        if (rank == 0 && tid == 0) {
            out[a] = token;
            if (token < 0)
                atomicOr(p.status, kStatusBadIndex);
        }
    } else {
        // ---- the drafts that stand, by every warp
        for (int j0 = 0; j0 < k; j0 += 32) {
            const int j = j0 + lane;
            bool good = false;
            if (j < k) {
                const int d = p.tokens[d0 + j];
                if (d >= 0 && d < V) {
                    const float x = value(target[(int64_t)(row0 + j) * p.target_stride + d]);
                    const float y = draft != nullptr ? value(draft[(int64_t)(d0 + j) * p.draft_stride + d]) : 1.f;
                    good = product_below(p.uniform[row0 + j], fmaxf(y, 0.f), fmaxf(x, 0.f));   // (NaN counts as 0)
                }
            }
            const unsigned m = __ballot_sync(0xffffffffu, good);
            a += m == 0xffffffffu ? 32 : __ffs(~m) - 1;
            if (m != 0xffffffffu)
                break;
        }
        Row<T> row;
        row.p = target + (int64_t)(row0 + a) * p.target_stride;
        row.q = a < k && draft != nullptr ? draft + (int64_t)(d0 + a) * p.draft_stride : nullptr;
        row.point = a < k && draft == nullptr ? p.tokens[d0 + a] : -1;
        const int tiles = (hi - lo + p.tile - 1) / p.tile;
        if (C > 1)
            cluster_wait_begun();
        for (int turn = 0;; ++turn) {
            // ---- the sums of this CTA's tiles, a tile to a warp
            for (int t = warp; t < tiles; t += kWarps) {
                const int t0 = lo + t * p.tile, t1 = min(hi, t0 + p.tile);
                const Sum w = row.q != nullptr ? row.template sum<true>(t0, t1, lane) : row.template sum<false>(t0, t1, lane);
                if (lane == 0)
                    tile_sum[t] = w;
            }
            __syncthreads();
            // ---- the sum over the row, the part that holds the wanted sum, and there the tile.  Where rounding leaves no sum
            // above it, the last part, tile and value with weight are taken
            const int each = (tiles + 31) / 32, f0 = min(tiles, lane * each), f1 = min(tiles, f0 + each);
            Sum before_run;      // what lies before this lane's run of tiles
            if (warp == 0) {
                Sum run = {0.f, 0.f};
                for (int t = f0; t < f1; ++t)
                    run = plus(run, tile_sum[t]);
                const Sum all = shfl(scan32(run, lane, 32, before_run), 31);
                if (lane < C) {
                    if (C > 1)
                        put_remote(&totals[rank], lane, ((unsigned long long)__float_as_uint(all.lo) << 32) | __float_as_uint(all.hi));
                    else
                        totals[0] = all;
                }
                __syncwarp();
            }
            if (C > 1)
                cluster_barrier();
            if (warp == 0) {
                const Sum t = lane < C ? totals[lane] : Sum{0.f, 0.f};
                Sum before;
                const Sum sum = scan32(t, lane, 8, before);
                const Sum all = shfl(sum, 7);
                // small sums are compared at a scale at which the product has its low part
                const float up = all.hi < 0x1p-64f ? 0x1p64f : 1.f;
                const Sum w = times(scaled(all, up), p.uniform[row0 + k]);
                const unsigned over = __ballot_sync(0xffffffffu, t.hi > 0.f && above(scaled(sum, up), w));
                const unsigned some = __ballot_sync(0xffffffffu, t.hi > 0.f);
                // (a sum past the range, which may have become infinite or NaN, draws nothing)
                const int who = !(all.hi < 0x1p127f) ? -1 : over != 0u ? __ffs(over) - 1 : some != 0u ? 31 - __clz(some) : -1;
                if (who == rank) {
                    // the lanes' runs, then the tiles of one run
                    Sum at = plus(shfl(before, who), before_run), last_at = at, first_at = at;
                    int first = -1, last = -1;
                    for (int i = f0; i < f1; ++i) {
                        const Sum v = tile_sum[i], next = plus(at, v);
                        if (v.hi > 0.f) {
                            last = i;
                            last_at = at;
                            if (first < 0 && above(scaled(next, up), w)) {
                                first = i;
                                first_at = at;
                            }
                        }
                        at = next;
                    }
                    const unsigned has = __ballot_sync(0xffffffffu, first >= 0), any = __ballot_sync(0xffffffffu, last >= 0);
                    const int l = has != 0u ? __ffs(has) - 1 : 31 - __clz(any);
                    const int tile = __shfl_sync(0xffffffffu, has != 0u ? first : last, l);
                    const Sum tile_at = shfl(has != 0u ? first_at : last_at, l);
                    if (lane == 0) {
                        chosen = tile;
                        start = tile_at;
                        want = w;
                        lift = up;
                        found = INT_MAX;
                        last_positive = -1;
                    }
                }
                if (lane == 0)
                    owner = who;
            }
            __syncthreads();
            if (owner < 0 && turn == 0 && a < k) {   // nothing is left of p_a: p_a itself
                row.q = nullptr;
                row.point = -1;
                if (C > 1)
                    cluster_barrier();   // (totals have been read by all)
                else
                    __syncthreads();
                continue;
            }
            if (owner < 0 && rank == 0 && tid == 0) {
                out[a] = -1;
                atomicOr(p.status, kStatusBadIndex);
            }
            if (owner != rank)
                break;
            // ---- the tile, kEach values to a thread at a time
            const int t0 = lo + chosen * p.tile, t1 = min(hi, t0 + p.tile);
            Sum run = start;
            const Sum w = want;
            const float up = lift;
            for (int i0 = t0; i0 < t1; i0 += kEach * kThreads) {
                const int i = i0 + kEach * tid;
                T x[kEach], y[kEach];
#pragma unroll
                for (int u = 0; u < kEach; ++u) {
                    x[u] = row.p[min(i + u, t1 - 1)];
                    if (row.q != nullptr)
                        y[u] = row.q[min(i + u, t1 - 1)];
                }
                Sum v[kEach], sum = {0.f, 0.f};
#pragma unroll
                for (int u = 0; u < kEach; ++u) {
                    v[u] = Sum{0.f, 0.f};
                    if (i + u < t1 && i + u != row.point)
                        v[u] = difference(value(x[u]), row.q != nullptr ? fmaxf(value(y[u]), 0.f) : 0.f);
                    sum = plus(sum, v[u]);
                }
                Sum before;
                const Sum incl = scan32(sum, lane, 32, before);
                if (lane == 31)
                    wscan[warp] = incl;
                __syncthreads();
                Sum before_warp;
                const Sum ws = scan32(lane < kWarps ? wscan[lane] : Sum{0.f, 0.f}, lane, kWarps, before_warp);
                Sum at = plus(plus(run, shfl(before_warp, warp)), before);
                int mine_first = INT_MAX, mine_last = -1;
#pragma unroll
                for (int u = 0; u < kEach; ++u) {
                    at = plus(at, v[u]);
                    if (v[u].hi > 0.f) {
                        mine_last = i + u;
                        if (mine_first == INT_MAX && above(scaled(at, up), w))
                            mine_first = i + u;
                    }
                }
                const int wfirst = __reduce_min_sync(0xffffffffu, mine_first), wlast = __reduce_max_sync(0xffffffffu, mine_last);
                if (lane == 0) {
                    if (wfirst != INT_MAX)
                        atomicMin(&found, wfirst);
                    if (wlast >= 0)
                        atomicMax(&last_positive, wlast);
                }
                run = plus(run, shfl(ws, kWarps - 1));
                __syncthreads();   // (wscan has been read)
            }
            if (tid == 0)
                out[a] = found != INT_MAX ? found : last_positive;
            break;
        }
    }
    if (rank == 0) {
        for (int j = tid; j < p.out_width; j += kThreads) {
            const int d = j < k ? p.tokens[d0 + j] : -1;
            if (j != a)
                out[j] = j < a ? d : -1;
            if (j < k && (d < 0 || d >= V))
                atomicOr(p.status, kStatusBadIndex);
        }
        if (tid == 0) {
            p.accepted[b] = a;
            if (p.seq != nullptr)
                p.seq_out[b] = p.seq[b] - (k - a);
        }
    }
}

}  // namespace

// CTAs per request: as many as are there at the same time, up to kMaxCluster, with kDeep values or more to a thread.  In us
// with 1, 2, 3, 4, 6 and 8: 48 mixed requests of 100277 39, 25, 19, 18, 16, 17; 160 of 128000 33, 27, 23, 31, 28, 46; 256 of
// 151937 77, 58, 63, 59, 63, 65.  One request of 32000 14, 13, 10, 11, 10, 11.  Few requests with wide vocabularies would take more:
// one of 151937 28, 21, 15, 14, 14, 11, sixteen 40, 25, 19, 18, 15, 14.
int verify_cluster_size(int num_reqs, int vocab, int sms)
{
    const int fit = std::min(kCtasPerSm * sms / std::max(1, num_reqs), vocab / (kDeep * kThreads));
    return std::max(1, std::min(fit, kMaxCluster));
}

// Values per tile: some 64 tiles to a CTA (four to a warp), between kMinTile and what the search looks at in one go
int verify_tile(int vocab, int cluster)
{
    const int part = (vocab + cluster - 1) / cluster;
    int tile = kMinTile;
    while ((tile < kEach * kThreads && part / tile > 64) || part / tile >= kMaxTiles)
        tile *= 2;
    return tile;
}

cudaError_t launch_verify(const VerifyParams &p, bool bf16, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.num_reqs * (unsigned)p.cluster);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster > 1 ? 2 : 1;
    const cudaError_t e = bf16 ? cudaLaunchKernelEx(&cfg, verify_kernel<__nv_bfloat16>, p) : cudaLaunchKernelEx(&cfg, verify_kernel<float>, p);
    if (e != cudaSuccess)
        (void)cudaGetLastError();
    return e;
}

}  // namespace dsv4
