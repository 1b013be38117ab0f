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
// What is decided next to a border has to be right, so the sums are held in about 48 bits: a weight is the exact
// difference of two floats as (high, low), and a thread's running sum is such a pair too (Knuth's two-sum); sums of tiles
// and the search are in 64 bits.  Products u q are exact there.
#include <cuda_bf16.h>
#include <limits.h>
#include <math.h>

#include "serving.h"

namespace dsv4 {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kTile = 1024;          // values per tile, or a multiple of it where a CTA's part has more than kMaxTiles
constexpr int kMaxTiles = 512;

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

__device__ __forceinline__ void add(Sum &s, float x)   // exact but for the rounding of the low parts' sum
{
    const float t = __fadd_rn(s.hi, x);
    const float b = __fsub_rn(t, s.hi);
    s.lo = __fadd_rn(s.lo, __fadd_rn(__fsub_rn(s.hi, __fsub_rn(t, b)), __fsub_rn(x, b)));
    s.hi = t;
}

// max(p - q, 0) of a value, exactly, into the sum
__device__ __forceinline__ void add_weight(Sum &s, float p, float q)
{
    const float d = __fsub_rn(p, q);
    if (!(d > 0.f))   // (the difference's sign is exact; NaN has no weight)
        return;
    const float b = __fsub_rn(d, p);
    const float e = __fsub_rn(__fsub_rn(p, __fsub_rn(d, b)), __fadd_rn(q, b));
    add(s, d);
    s.lo = __fadd_rn(s.lo, e);
}

// A request's row of weights: p, less the draft's q, or without the drafted token
template <typename T>
struct Row {
    const T *p, *q;
    int point;         // this value has no weight (-1: none)
    __device__ __forceinline__ void load(int i, float &x, float &y) const
    {
        x = value(p[i]);
        y = q != nullptr ? fmaxf(value(q[i]), 0.f) : 0.f;   // (NaN: 0)
    }
    __device__ __forceinline__ double weight(int i) const
    {
        float x, y;
        load(i, x, y);
        const double d = (double)x - (double)y;
        return d > 0.0 && i != point ? d : 0.0;
    }
};

template <typename T>
__global__ void __launch_bounds__(kThreads) verify_kernel(const VerifyParams p)
{
    __shared__ double tile_sum[kMaxTiles];
    __shared__ double totals[kMaxCluster];                    // the cluster's parts of the row
    __shared__ unsigned long long bests[2][kMaxCluster];      // greedy: (order key of the value, ~index)
    __shared__ unsigned long long wbest[kWarps];
    __shared__ double wscan[kWarps];
    __shared__ int found, last_positive, chosen;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = p.cluster, b = blockIdx.x / C;
    const uint32_t rank = C > 1 ? cluster_rank() : 0u;
    auto sync_all = [&]() {
        if (C > 1)
            cluster_barrier();
        else
            __syncthreads();
    };
    const T *target = static_cast<const T *>(p.target), *draft = static_cast<const T *>(p.draft);
    const int V = p.vocab;
    griddep_wait();
    griddep_launch();

    const int base = p.start[0], row0 = p.start[b] - base, rows = p.start[b + 1] - p.start[b];
    const int d0 = row0 - b, k = rows - 1;   // (every request before this one has a row more than drafts)
    int32_t *out = p.out + (int64_t)b * p.out_stride;
    const bool ok = rows >= 1 && rows <= p.num_rows && row0 >= 0 && row0 <= p.num_rows - rows && d0 >= 0 && d0 <= p.num_drafts - k &&
                    rows <= p.out_width;
    if (!ok) {   // (the same in every CTA of the cluster)
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
    const int lo = min(V, (int)rank * part), hi = min(V, lo + part);

    int a = 0;
    int token = -1;      // of a greedy request
    if (greedy) {
        for (int j = 0;; ++j) {   // row j: its largest value, the lowest index of equal ones
            const T *row = target + (int64_t)(row0 + j) * p.target_stride;
            float best = -INFINITY;
            int at = INT_MAX;
            constexpr int kDeep = 8;
            for (int i0 = lo; i0 < hi; i0 += kDeep * kThreads) {
                float x[kDeep];
#pragma unroll
                for (int u = 0; u < kDeep; ++u) {
                    const int i = i0 + u * kThreads + tid;
                    x[u] = i < hi ? value(row[i]) : -INFINITY;
                }
#pragma unroll
                for (int u = 0; u < kDeep; ++u) {
                    const int i = i0 + u * kThreads + tid;
                    if (i < hi && (x[u] > best || (x[u] == best && at == INT_MAX))) {
                        best = x[u];
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
            if (j == k || token != p.tokens[d0 + j])
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
        bool bad = false;
        for (int j0 = 0; j0 < k; j0 += 32) {
            const int j = j0 + lane;
            bool good = false;
            if (j < k) {
                const int d = p.tokens[d0 + j];
                if (d >= 0 && d < V) {
                    const float x = value(target[(int64_t)(row0 + j) * p.target_stride + d]);
                    const float y = draft != nullptr ? value(draft[(int64_t)(d0 + j) * p.draft_stride + d]) : 1.f;
                    good = (double)p.uniform[row0 + j] * (double)y < (double)x;
                } else {
                    bad = true;
                }
            }
            const unsigned m = __ballot_sync(0xffffffffu, good);
            a += m == 0xffffffffu ? 32 : __ffs(~m) - 1;
            if (m != 0xffffffffu)
                break;
        }
        if (bad)
            atomicOr(p.status, kStatusBadIndex);
        const double u = p.uniform[row0 + k];
        Row<T> row;
        row.p = target + (int64_t)(row0 + a) * p.target_stride;
        row.q = a < k && draft != nullptr ? draft + (int64_t)(d0 + a) * p.draft_stride : nullptr;
        row.point = a < k && draft == nullptr ? p.tokens[d0 + a] : -1;
        for (int turn = 0;; ++turn) {
            // ---- the sums of this CTA's tiles, a tile to a warp
            const int tiles = (hi - lo + p.tile - 1) / p.tile;
            for (int t = warp; t < tiles; t += kWarps) {
                const int t0 = lo + t * p.tile, t1 = min(hi, t0 + p.tile);
                Sum s = {0.f, 0.f};
                for (int i0 = t0; i0 < t1; i0 += 256) {
                    float x[8], y[8];
#pragma unroll
                    for (int v = 0; v < 8; ++v) {
                        const int i = i0 + 32 * v + lane;
                        x[v] = y[v] = 0.f;
                        if (i < t1)
                            row.load(i, x[v], y[v]);
                        if (i == row.point)
                            x[v] = 0.f;
                    }
#pragma unroll
                    for (int v = 0; v < 8; ++v)
                        add_weight(s, x[v], y[v]);
                }
                double w = (double)s.hi + (double)s.lo;
#pragma unroll
                for (int d = 16; d > 0; d >>= 1)
                    w += __shfl_xor_sync(0xffffffffu, w, d);
                if (lane == 0)
                    tile_sum[t] = w;
            }
            __syncthreads();
            // ---- the row's sum, and what comes before this CTA's part: every warp the same
            double mine = 0.0;
            for (int t0 = 0; t0 < tiles; t0 += 32) {
                double w = t0 + lane < tiles ? tile_sum[t0 + lane] : 0.0;
#pragma unroll
                for (int d = 16; d > 0; d >>= 1)
                    w += __shfl_xor_sync(0xffffffffu, w, d);
                mine += w;
            }
            if (tid < C) {
                if (C > 1)
                    put_remote(&totals[rank], tid, (unsigned long long)__double_as_longlong(mine));
                else
                    totals[0] = mine;
            }
            sync_all();
            double all = 0.0, before = 0.0;
            int last = -1;       // the last part that has weight
            for (int r = 0; r < C; ++r) {
                before += r < (int)rank ? totals[r] : 0.0;
                all += totals[r];
                last = totals[r] > 0.0 ? r : last;
            }
            if (last < 0 && turn == 0 && a < k) {   // nothing is left of p_a: p_a itself
                row.q = nullptr;
                row.point = -1;
                sync_all();      // (totals have been read by all)
                continue;
            }
            if (last < 0) {
                if (rank == 0 && tid == 0) {
                    out[a] = -1;
                    atomicOr(p.status, kStatusBadIndex);
                }
                break;
            }
            const double want = u * all;
            // the first part, tile and value whose sum is above `want`; where rounding leaves none, the last ones with weight
            double at = 0.0;
            int owner = last;
            for (int r = 0; r <= last; ++r) {
                if (at + totals[r] > want) {
                    owner = r;
                    break;
                }
                at += totals[r];
            }
            if (owner != (int)rank)
                break;
            if (warp == 0) {
                int tile = -1, tail = -1;
                double run = before, start = before, tail_start = before;
                for (int t0 = 0; t0 < tiles && tile < 0; t0 += 32) {
                    const double w = t0 + lane < tiles ? tile_sum[t0 + lane] : 0.0;
                    double incl = w;
#pragma unroll
                    for (int d = 1; d < 32; d <<= 1) {
                        const double y = __shfl_up_sync(0xffffffffu, incl, d);
                        if (lane >= d)
                            incl += y;
                    }
                    const unsigned above = __ballot_sync(0xffffffffu, w > 0.0 && run + incl > want);
                    const unsigned some = __ballot_sync(0xffffffffu, w > 0.0);
                    if (above != 0u) {
                        const int l = __ffs(above) - 1;
                        tile = t0 + l;
                        start = __shfl_sync(0xffffffffu, run + (incl - w), l);
                    }
                    if (some != 0u) {
                        const int l = 31 - __clz(some);
                        tail = t0 + l;
                        tail_start = __shfl_sync(0xffffffffu, run + (incl - w), l);
                    }
                    run += __shfl_sync(0xffffffffu, incl, 31);
                }
                if (lane == 0) {
                    chosen = tile >= 0 ? tile : tail;
                    wscan[0] = tile >= 0 ? start : tail_start;
                    found = INT_MAX;
                    last_positive = -1;
                }
            }
            __syncthreads();
            const int t0 = lo + chosen * p.tile, t1 = min(hi, t0 + p.tile);
            double run = wscan[0];
            // ---- the tile, two values to a thread at a time
            for (int i0 = t0; i0 < t1; i0 += 2 * kThreads) {
                const int i = i0 + 2 * tid;
                const double w0 = i < t1 ? row.weight(i) : 0.0, w1 = i + 1 < t1 ? row.weight(i + 1) : 0.0;
                double incl = w0 + w1;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const double y = __shfl_up_sync(0xffffffffu, incl, d);
                    if (lane >= d)
                        incl += y;
                }
                __syncthreads();   // (wscan has been read)
                if (lane == 31)
                    wscan[warp] = incl;
                __syncthreads();
                double pre = run + (incl - (w0 + w1));
                for (int w = 0; w < kWarps; ++w) {
                    if (w < warp)
                        pre += wscan[w];
                    run += wscan[w];
                }
                if (w0 > 0.0 && pre + w0 > want)
                    atomicMin(&found, i);
                else if (w1 > 0.0 && pre + w0 + w1 > want)
                    atomicMin(&found, i + 1);
                if (w0 > 0.0 || w1 > 0.0)
                    atomicMax(&last_positive, w1 > 0.0 ? i + 1 : i);
            }
            __syncthreads();
            if (tid == 0)
                out[a] = found != INT_MAX ? found : last_positive;
            break;
        }
    }
    if (rank == 0) {
        for (int j = tid; j < p.out_width; j += kThreads)
            if (j != a)
                out[j] = j < a ? p.tokens[d0 + j] : -1;
        if (tid == 0) {
            p.accepted[b] = a;
            if (p.seq != nullptr)
                p.seq_out[b] = p.seq[b] - (k - a);
        }
    }
}

}  // namespace

// CTAs per request: as many as there are for it, with four tiles or more to each
int verify_cluster_size(int num_reqs, int vocab, int sms)
{
    int c = 1;
    while (c < kMaxCluster && 2ll * c * num_reqs <= 2 * sms && 2 * c * 4 * kTile <= vocab)
        c *= 2;
    return c;
}

int verify_tile(int vocab, int cluster)
{
    const int part = (vocab + cluster - 1) / cluster;
    return kTile * ((part + kTile * kMaxTiles - 1) / (kTile * kMaxTiles));
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
