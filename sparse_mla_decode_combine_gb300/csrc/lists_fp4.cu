// lists_fp4.cu -- a kernel of its own for the lists of cache slots (lists_fp4.cuh), one CTA per token: for decodes whose
// CTAs take runs of the blocks of many tokens, and so need every token's length before they begin.
//
// A token without a key gets its outputs here: zeros, and the sink (or -inf) as its lse.
#include <algorithm>
#include <cmath>

#include "lists_fp4.cuh"

namespace dsv4 {
namespace {

constexpr int kThreads = 512;
constexpr int kLoads = 4;   // entries of a row that a thread has in flight: 2048 in all

struct SyncAll {
    __device__ __forceinline__ void operator()() const { __syncthreads(); }
    __device__ __forceinline__ bool any(bool v) const { return __syncthreads_or(v); }
};

__global__ void __launch_bounds__(kThreads) lists_fp4_kernel(const Lists4Params p)
{
    griddep_wait();
    griddep_launch();   // (the decode waits for this grid itself)
    extern __shared__ unsigned long long tab[];
    __shared__ int wsum[kLoads * kThreads / 32];
    const int t = blockIdx.x, tid = threadIdx.x;
    if (tid < p.groups)
        p.joins[tid * gridDim.x + t] = make_int2(0, 0);
    const int len = lists::build<kThreads, kLoads>(p, t, tid, tab, wsum, SyncAll(), [](int len) { return make_int2(0, len); });
    if (tid == 0)
        p.lens[t] = len;
    if (len == 0) {
        for (int i = tid; i < p.num_heads * kLatent / 8; i += kThreads)
            *reinterpret_cast<uint4 *>(p.out + (int64_t)t * p.num_heads * kLatent + 8 * i) = make_uint4(0, 0, 0, 0);
        if (p.lse != nullptr && tid < p.num_heads)
            p.lse[(int64_t)t * p.num_heads + tid] = p.sink != nullptr ? p.sink[tid] : -INFINITY;
    }
}

// The lists with their positions, for a kernel that returns something per key.  The CTAs of a token share its window's part (the
// top-k part is made by each of them, the same).
__global__ void __launch_bounds__(kThreads) lists_positions_kernel(const Lists4Params p)
{
    griddep_wait();
    griddep_launch();   // (the next kernel waits for this grid itself)
    extern __shared__ unsigned long long tab[];
    __shared__ int wsum[kLoads * kThreads / 32];
    const int t = blockIdx.x, part = blockIdx.y, parts = gridDim.y;
    const int len = lists::build<kThreads, kLoads, true>(p, t, threadIdx.x, tab, wsum, SyncAll(), [&](int len) {
        return make_int2((int)((long long)len * part / parts), (int)((long long)len * (part + 1) / parts));
    });
    if (part > 0)
        return;
    bool later = false;
    if (p.req_idx != nullptr) {
        const int r = p.req_idx[t];
        for (int i = threadIdx.x; i < t; i += kThreads)
            later |= p.req_idx[i] == r && p.seq_lens[i] > 0;
    }
    later = __syncthreads_or(later);
    if (threadIdx.x == 0) {
        p.lens[t] = len;
        p.later[t] = later ? 1 : 0;
    }
}

}  // namespace

cudaError_t launch_lists_positions(const Lists4Params &p, int sms, cudaStream_t stream)
{
    const cudaError_t e = set_smem_once(reinterpret_cast<const void *>(lists_positions_kernel), p.smem_bytes, kAttrPositions);
    if (e != cudaSuccess)
        return e;
    // (one CTA makes 2048 entries of a window in 4 us, 30000 in 17)
    const int parts = std::max(1, std::min((p.window + 2047) / 2048, 2 * sms / p.num_tokens));
    return launch_dependent(lists_positions_kernel, dim3((unsigned)p.num_tokens, (unsigned)parts), kThreads, (size_t)p.smem_bytes,
                            stream, p);
}

cudaError_t launch_lists_fp4(const Lists4Params &p, cudaStream_t stream)
{
    if (p.num_tokens <= 0)
        return cudaSuccess;
    const cudaError_t e = set_smem_once(reinterpret_cast<const void *>(lists_fp4_kernel), p.smem_bytes, kAttrFp4Lists);
    if (e != cudaSuccess)
        return e;
    return launch_dependent(lists_fp4_kernel, dim3((unsigned)p.num_tokens), kThreads, (size_t)p.smem_bytes, stream, p);
}

}  // namespace dsv4
