// decode_fp4.cu -- sparse-MLA decode over the 4-bit cache, plain form: one CTA per (token, eight
// heads), one warp per head, 32 keys at a time dequantised to fp32 in shared memory, an online softmax.
//   s_p = scale * q . k_p (576 dims), lse = ln(sum_p e^{s_p} + e^{sink}), out = sum_p e^{s_p - lse} v_p
// over the token's combined list (positions), each position through the block table to its entry.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fp4.h"

namespace dsv4 {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 32;
constexpr int kPitch = kDim + 1;
constexpr int kSmemBytes = (kTile * kPitch + kWarps * kDim) * 4;

__device__ __forceinline__ float scale_of(unsigned b)   // UE8M0
{
    if (b == 0xFFu)
        return __int_as_float(0x7FC00000);
    return b == 0u ? 0x1p-127f : __int_as_float((int)(b << 23));
}

__device__ __forceinline__ float e2m1(unsigned code)
{
    const unsigned m = code & 7u;
    // (a code's bits at the top of an fp32 exponent and mantissa are its value times 2^-126)
    const float v = __int_as_float((int)(m << 22)) * 0x1p126f;
    return code & 8u ? -v : v;
}

__device__ __forceinline__ float bf16(unsigned bits) { return __int_as_float((int)(bits << 16)); }

__global__ void __launch_bounds__(kThreads) decode_fp4_kernel(const Decode4Params p)
{
    extern __shared__ float sm[];
    __shared__ int ok[kTile];
    float *key = sm, *q = sm + kTile * kPitch;
    const int groups = p.num_heads / kWarps;
    const int t = blockIdx.x / groups, h = blockIdx.x % groups * kWarps + (threadIdx.x >> 5);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int d = lane; d < kDim; d += 32)
        q[warp * kDim + d] = bf16(p.q[t * p.q_token_stride + (int64_t)h * kDim + d]);
    const int row = p.req_idx ? p.req_idx[t] : t;
    const bool row_ok = row >= 0 && row < p.num_reqs;
    const int n = p.lens[t];
    if (!row_ok && n > 0 && threadIdx.x == 0)
        atomicOr(p.status, kStatusBadIndex);
    float m = -INFINITY, l = 0.f, acc[16] = {};
    for (int k0 = 0; k0 < n; k0 += kTile) {
        __syncthreads();
        for (int k = warp; k < kTile; k += kWarps) {
            int64_t slot = -1;
            if (row_ok && k0 + k < n) {
                const int pos = p.lists[(int64_t)t * p.list_w + k0 + k], blk = pos / p.page;
                const int phys = blk < p.max_blocks ? p.block_table[row * p.bt_stride + blk] : -1;
                if (phys >= 0 && phys < p.num_blocks)
                    slot = (int64_t)phys * p.page + pos % p.page;
                else
                    atomicOr(p.status, kStatusBadIndex);
            }
            if (lane == 0)
                ok[k] = slot >= 0;
            const uint8_t *e = p.kv + slot * kEntry4Bytes;
            for (int d = lane; d < kDim; d += 32) {
                float v = 0.f;
                if (slot >= 0)
                    v = d < kLatent ? e2m1(e[d >> 1] >> (4 * (d & 1))) * scale_of(e[kScale4Offset + d / kScale4Block])
                                    : bf16(reinterpret_cast<const uint16_t *>(e + kRope4Offset)[d - kLatent]);
                key[k * kPitch + d] = v;
            }
        }
        __syncthreads();
        float s = 0.f;
        for (int d = 0; d < kDim; ++d)
            s = fmaf(q[warp * kDim + d], key[lane * kPitch + d], s);
        s = ok[lane] ? s * p.scale : -INFINITY;
        float mb = s;
        for (int o = 16; o > 0; o >>= 1)
            mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, o));
        const float mn = fmaxf(m, mb);
        if (mn == -INFINITY && !__any_sync(0xffffffffu, isnan(s)))
            continue;
        const float w = ok[lane] ? expf(s - mn) : 0.f;
        const float a = expf(m - mn);
        float ws = w;
        for (int o = 16; o > 0; o >>= 1)
            ws += __shfl_xor_sync(0xffffffffu, ws, o);
        l = l * a + ws;
        m = mn;
        for (int i = 0; i < 16; ++i)
            acc[i] *= a;
        for (int k = 0; k < kTile; ++k) {
            const float wk = __shfl_sync(0xffffffffu, w, k);
            if (wk != 0.f)
                for (int i = 0; i < 16; ++i)
                    acc[i] = fmaf(wk, key[k * kPitch + lane + 32 * i], acc[i]);
        }
    }
    const float sk = p.sink ? p.sink[h] : -INFINITY;
    const float M = fmaxf(m, sk);
    const float z = M == -INFINITY ? 0.f : l * expf(m - M) + expf(sk - M);
    const float f = z > 0.f && m != -INFINITY ? expf(m - M) / z : 0.f;
    const int64_t o = (int64_t)t * p.num_heads + h;
    for (int i = 0; i < 16; ++i) {
        const __nv_bfloat16 b = __float2bfloat16_rn(acc[i] * f);
        p.out[o * kLatent + lane + 32 * i] = *reinterpret_cast<const uint16_t *>(&b);
    }
    if (lane == 0 && p.lse)
        p.lse[o] = z > 0.f ? M + logf(z) : -INFINITY;
}

}  // namespace

cudaError_t launch_decode_fp4(const Decode4Params &p, cudaStream_t stream)
{
    if (p.num_tokens <= 0)
        return cudaSuccess;
    cudaError_t e = set_smem_once(reinterpret_cast<const void *>(decode_fp4_kernel), kSmemBytes, kAttrFp4);
    if (e != cudaSuccess)
        return e;
    decode_fp4_kernel<<<p.num_tokens * (p.num_heads / kWarps), kThreads, kSmemBytes, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace dsv4
