// key_weights.cu -- the attention weight that a decode step gave each key, added up per cache row and position.
//
//   weights[row][p] += sum_h e^{scale q_h . k_p - lse_h}     for the keys p of each token's list
// with the lse that the decode returned (its sink counts there).  Tokens of one row are added in ascending order, one
// rounding each, so the result does not depend on timing.
#include <math.h>

#include "serving.h"
#include "tcgen05.cuh"

namespace dsv4 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kKeys = 16;
constexpr int kAddThreads = 512;
constexpr int kAddSlices = 16;

__device__ __forceinline__ float key_value(const uint8_t *e, int entry_bytes, int d)
{
    if (entry_bytes == kEntry4Bytes) {
        if (d >= kLatent)
            return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(e + kRope4Offset)[d - kLatent] << 16);
        const uint32_t c = (e[d >> 1] >> (4 * (d & 1))) & 15u, se = e[kScale4Offset + d / kScale4Block];
        const float m = (c & 7u) < 2u ? 0.5f * (float)(c & 1u) : ldexpf(1.f + 0.5f * (float)(c & 1u), (int)((c >> 1) & 3u) - 1);
        return (c & 8u ? -m : m) * (se == 255u ? NAN : ldexpf(1.f, (int)se - 127));
    }
    if (d >= kLatent)
        return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(e + kRopeOffset)[d - kLatent] << 16);
    const uint32_t c = e[d], se = e[kScaleOffset + d / kScaleBlock], x = (c >> 3) & 15u, f = c & 7u;
    const float m = (c & 127u) == 127u ? NAN : x == 0u ? ldexpf((float)f, -9) : ldexpf(1.f + 0.125f * (float)f, (int)x - 7);
    return (c & 128u ? -m : m) * (se == 255u ? NAN : ldexpf(1.f, (int)se - 127));
}

__global__ void __launch_bounds__(kThreads) key_weights_kernel(const KeyWeightsParams p)
{
    __shared__ float keys[kKeys][kDim];
    __shared__ float sums[kWarps][kKeys];
    griddep_wait();
    griddep_launch();
    const int t = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int len = __ldcg(p.lens + t);
    for (int k0 = blockIdx.x * kKeys; k0 < len; k0 += gridDim.x * kKeys) {
        for (int i = tid; i < kKeys * kDim; i += kThreads) {
            const int k = i / kDim, d = i % kDim;
            const int slot = k0 + k < len ? __ldcg(p.slots + (int64_t)t * p.list_w + k0 + k) : -1;
            keys[k][d] = slot >= 0 ? key_value(p.kv + (int64_t)slot * p.entry_bytes, p.entry_bytes, d) : 0.f;
        }
        __syncthreads();
        float mine = 0.f;   // lane k: the sum of key k over this warp's heads
        for (int h = warp; h < p.num_heads; h += kWarps) {
            const uint16_t *q = p.q + (int64_t)t * p.q_token_stride + h * kDim;
            float dot[kKeys];
#pragma unroll
            for (int k = 0; k < kKeys; ++k)
                dot[k] = 0.f;
            for (int d = lane; d < kDim; d += 32) {
                const float x = __uint_as_float((uint32_t)q[d] << 16);
#pragma unroll
                for (int k = 0; k < kKeys; ++k)
                    dot[k] = fmaf(x, keys[k][d], dot[k]);
            }
            float l = p.lse[(int64_t)t * p.num_heads + h];
            if (l == -INFINITY)
                l = INFINITY;
#pragma unroll
            for (int k = 0; k < kKeys; ++k) {
                float s = dot[k];
#pragma unroll
                for (int d = 16; d > 0; d >>= 1)
                    s += __shfl_xor_sync(0xffffffffu, s, d);
                if (lane == k)
                    mine += expf(fmaf(s, p.scale, -l));
            }
        }
        if (lane < kKeys)
            sums[warp][lane] = mine;
        __syncthreads();
        if (tid < kKeys && k0 + tid < len) {
            float s = 0.f;
            for (int w = 0; w < kWarps; ++w)
                s += sums[w][tid];
            __stcg(p.got + (int64_t)t * p.list_w + k0 + tid, s);
        }
        __syncthreads();
    }
}

// A row's tokens, one after the other; positions are dealt out to the slices in runs of 256.
__global__ void __launch_bounds__(kAddThreads) add_weights_kernel(const KeyWeightsParams p)
{
    griddep_wait();
    griddep_launch();
    const int r = blockIdx.y, slice = blockIdx.x, tid = threadIdx.x;
    float *row = p.weights + (int64_t)r * p.weights_stride;
    for (int t = 0; t < p.num_tokens; ++t) {
        if ((p.req_idx != nullptr ? p.req_idx[t] : t) != r)
            continue;
        const int len = __ldcg(p.lens + t);
        for (int i = tid; i < len; i += kAddThreads) {
            const int pos = __ldcg(p.positions + (int64_t)t * p.list_w + i);
            if ((pos >> 8) % kAddSlices == slice && __ldcg(p.slots + (int64_t)t * p.list_w + i) >= 0)
                row[pos] += __ldcg(p.got + (int64_t)t * p.list_w + i);
        }
        __syncthreads();   // the next token's sums come on top
    }
}

}  // namespace

cudaError_t launch_key_weights(const KeyWeightsParams &p, int sms, cudaStream_t stream)
{
    const unsigned blocks = (unsigned)max(1, min((p.list_w + kKeys - 1) / kKeys, 256));
    const cudaError_t e = launch_dependent(key_weights_kernel, dim3(blocks, (unsigned)p.num_tokens), kThreads, 0, stream, p);
    if (e != cudaSuccess)
        return e;
    return launch_dependent(add_weights_kernel, dim3(kAddSlices, (unsigned)p.num_reqs), kAddThreads, 0, stream, p);
}

}  // namespace dsv4
