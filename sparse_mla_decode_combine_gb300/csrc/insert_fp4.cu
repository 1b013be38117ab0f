// insert_fp4.cu -- norms of the queries (per head) and of the key, GPT-J rotation of both, and the
// 4-bit insert of the key, in one pass:
//   q_out[t][h] = RoPE_pos(q[t][h] / sqrt(mean(q[t][h]^2) + eps) * w_q)        (576 dims, one rounding)
//   k[t]        = RoPE_pos(kv[t] with its first n dims divided by sqrt(mean of their squares + eps), times w_kv)
//   entry(k):     per 32 latent values the smallest UE8M0 exponent e with 6 * 2^e >= amax (0 for amax 0,
//                 clamped to [-127, 125]), E2M1 codes of k * 2^-e (nearest, ties to even), BF16 rope
//   k_out[t]    = the values that the entry stands for, in BF16
// The rotation turns the interleaved pairs (512 + 2i, 513 + 2i) by the angle whose cosine and sine
// are cos_sin[pos][i] and cos_sin[pos][32 + i].
//
// Arithmetic.  Queries: fp32, one rounding to BF16.  The key's codes are those of the exactly computed
// key: a 4-bit step is a quarter of the value or more, so a value that fp32 puts on the wrong side of a
// rounding border would be off by all of it.  The sum of squares and the root are taken in fp64 (BF16
// squares are exact there); the values themselves in fp32, with a check whether any value of the entry
// lies within 2^-21 of a border of its code or its block's exponent; the few tokens that have one
// (about one in seven hundred) repeat the quantisation in fp64.
//
// One CTA per token: warps 0..15 take the query heads, four at a time (their loads all in flight
// before any use), lane l holding the BF16 pairs l + 32 j (j < 9; j = 8 is the rope part, pair i = l)
// so a pair never leaves its lane; warp 16 builds the entry, half a warp to a block of 32 values.
#include <cuda_bf16.h>
#include <cuda_fp4.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fp4.h"

namespace dsv4 {
namespace {

constexpr int kQWarps = 16;
constexpr int kHeadsIter = 4;      // heads a warp has in flight at once
constexpr int kThreads = 32 * (kQWarps + 1);
constexpr int kPairs = kDim / 2;   // 288 BF16 pairs per head; pairs 256.. are the rope part
constexpr float kNear = 1.f / (1 << 21);

__device__ __forceinline__ float2 unpack_bf16x2(uint32_t v)
{
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}

__device__ __forceinline__ uint32_t pack_rn_bf16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ double warp_sum(double v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <typename T>
__device__ __forceinline__ T half_warp_max(T v)
{
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
        const T u = __shfl_xor_sync(0xffffffffu, v, o);
        v = u > v ? u : v;
    }
    return v;
}

// Smallest integer e with 6 * 2^e >= amax (0 for amax 0), clamped to [-127, 125].  For amax in
// [2^k, 2^(k+1)) the answer is k - 2 or k - 1; one exact comparison decides.
__device__ __forceinline__ int exponent_of(float amax)
{
    if (!(amax > 0.f))
        return 0;
    if (amax > 1.5f * 0x1p127f)   // past 6 * 2^125
        return 125;
    int e = ilogbf(amax) - 2;
    if (ldexpf(6.f, e) < amax)
        ++e;
    return e < -127 ? -127 : e;
}

__device__ __forceinline__ int exponent_of(double amax)
{
    if (!(amax > 0.0))
        return 0;
    if (amax > 1.5 * 0x1p127)
        return 125;
    int e = ilogb(amax) - 2;
    if (ldexp(6.0, e) < amax)
        ++e;
    return e < -127 ? -127 : e;
}

__device__ __forceinline__ float pow2f(int e)   // 2^e, -126 <= e <= 127
{
    return __int_as_float((e + 127) << 23);
}

// two E2M1 codes, the first value's in the low half (nearest, ties to even, past 6 -> 6; NaN -> 6)
__device__ __forceinline__ uint32_t codes_of(float a, float b)
{
    return __nv_cvt_float2_to_fp4x2(make_float2(a, b), __NV_E2M1, cudaRoundNearest);
}

__device__ __forceinline__ uint32_t code_of(double t)
{
    const double a = fabs(t);
    uint32_t c = 7u;
    if (a <= 5.0)   // the borders of the codes 0, 1/2, 1, 3/2, 2, 3, 4, 6; a border goes to the even code
        c = a <= 0.25 ? 0u : a < 0.75 ? 1u : a <= 1.25 ? 2u : a < 1.75 ? 3u : a <= 2.5 ? 4u : a < 3.5 ? 5u : 6u;
    return c | (signbit(t) && !isnan(t) ? 8u : 0u);
}

__device__ __forceinline__ float value_of(uint32_t code)
{
    const float m = (code & 6u) == 0u ? 0.5f * (float)(code & 1u)
                                      : (1.f + 0.5f * (float)(code & 1u)) * pow2f((int)((code >> 1) & 3u) - 1);
    return code & 8u ? -m : m;
}

__global__ void __launch_bounds__(kThreads) qk_norm_rope_kv_insert_fp4_kernel(const Insert4Params p)
{
    const int t = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t pos = p.positions[t];
    const bool rot = pos >= 0 && pos < p.max_pos;
    float c = 1.f, s = 0.f;   // this lane's rope pair i = lane
    if (rot) {
        c = __ldg(p.cos_sin + pos * 64 + lane);
        s = __ldg(p.cos_sin + pos * 64 + 32 + lane);
    } else if (threadIdx.x == 0) {
        atomicOr(p.status, kStatusBadIndex);
    }

    if (warp < kQWarps) {
        float w[18];   // the norm weight of this lane's 18 dims (pairs lane + 32 j)
#pragma unroll
        for (int j = 0; j < 9; ++j) {
            const int d = 2 * (lane + 32 * j);
            w[2 * j] = p.q_w ? __ldg(p.q_w + d) : 1.f;
            w[2 * j + 1] = p.q_w ? __ldg(p.q_w + d + 1) : 1.f;
        }
        for (int h0 = warp; h0 < p.num_heads; h0 += kHeadsIter * kQWarps) {
            uint32_t x[kHeadsIter][9];
#pragma unroll
            for (int k = 0; k < kHeadsIter; ++k) {   // every head's loads in flight before any use
                const int h = h0 + k * kQWarps;
                const uint32_t *a = p.q + t * p.q_stride + (int64_t)h * kPairs;
#pragma unroll
                for (int j = 0; j < 9; ++j)
                    x[k][j] = h < p.num_heads ? __ldg(a + lane + 32 * j) : 0u;
            }
#pragma unroll
            for (int k = 0; k < kHeadsIter; ++k) {
                const int h = h0 + k * kQWarps;
                if (h >= p.num_heads)
                    break;
                float ss = 0.f;
#pragma unroll
                for (int j = 0; j < 9; ++j) {
                    const float2 v = unpack_bf16x2(x[k][j]);
                    ss = fmaf(v.x, v.x, fmaf(v.y, v.y, ss));
                }
                ss = warp_sum(ss);
                const float r = 1.f / sqrtf(ss / (float)kDim + (float)p.eps);
                uint32_t *o = p.q_out + t * p.q_out_stride + (int64_t)h * kPairs;
#pragma unroll
                for (int j = 0; j < 9; ++j) {
                    const float2 v = unpack_bf16x2(x[k][j]);
                    float y0 = v.x * r * w[2 * j], y1 = v.y * r * w[2 * j + 1];
                    if (j == 8) {
                        const float u0 = y0 * c - y1 * s;
                        const float u1 = y0 * s + y1 * c;
                        y0 = u0;
                        y1 = u1;
                    }
                    o[lane + 32 * j] = pack_rn_bf16x2(y0, y1);
                }
            }
        }
        return;
    }

    // ---- warp 16: the token's key
    const int64_t slot = p.slots[t];
    if (lane == 0 && slot >= p.num_slots)
        atomicOr(p.status, kStatusBadIndex);
    const bool write = slot >= 0 && slot < p.num_slots && rot;
    uint32_t x[9];
#pragma unroll
    for (int j = 0; j < 9; ++j)
        x[j] = __ldg(p.kv + t * p.kv_stride + lane + 32 * j);
    const int nj = p.kv_norm_dims / 64;   // pairs lane + 32 j with j < nj are normalised
    double root = 1.0;
    if (nj > 0) {
        double ss = 0.0;
#pragma unroll
        for (int j = 0; j < 9; ++j) {
            const float2 v = unpack_bf16x2(x[j]);
            if (j < nj)
                ss = fma((double)v.x, (double)v.x, fma((double)v.y, (double)v.y, ss));
        }
        root = sqrt(warp_sum(ss) / (double)p.kv_norm_dims + p.eps);
    }
    const float r = (float)(1.0 / root);
    float2 y[9];
    float2 w[9];
#pragma unroll
    for (int j = 0; j < 9; ++j) {
        const bool normed = j < nj;
        const int d = 2 * (lane + 32 * j);
        w[j] = make_float2(1.f, 1.f);
        if (normed && p.kv_w)
            w[j] = make_float2(__ldg(p.kv_w + d), __ldg(p.kv_w + d + 1));
        const float2 v = unpack_bf16x2(x[j]);
        y[j] = normed ? make_float2(v.x * r * w[j].x, v.y * r * w[j].y) : v;
    }
    int ex[8];
    uint32_t code[8];
    bool near = false;   // some value or block maximum lies next to a border
#pragma unroll
    for (int j = 0; j < 8; ++j) {   // blocks 2 j (lanes 0..15) and 2 j + 1 (lanes 16..31)
        const float a0 = fabsf(y[j].x), a1 = fabsf(y[j].y);
        const float amax = half_warp_max(fmaxf(fmaxf(a0, a1), 0.f));   // (a NaN counts as 0)
        ex[j] = exponent_of(amax);
        const float f = pow2f(-ex[j]);
        const float t0 = y[j].x * f, t1 = y[j].y * f;
        code[j] = codes_of(t0, t1);
        if (nj > 0) {
            near |= exponent_of(amax * (1.f - kNear)) != exponent_of(amax * (1.f + kNear)) ||
                    (amax < 0x1p-100f && amax > 0.f);
            near |= codes_of(t0 * (1.f - kNear), t1 * (1.f - kNear)) != codes_of(t0 * (1.f + kNear), t1 * (1.f + kNear));
        }
    }
    if (__any_sync(0xffffffffu, near)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 v = unpack_bf16x2(x[j]);
            const double y0 = (double)v.x / root * (double)w[j].x, y1 = (double)v.y / root * (double)w[j].y;
            const double a0 = fabs(y0), a1 = fabs(y1);
            double a = a0 > a1 || isnan(a1) ? a0 : a1;
            a = isnan(a) ? 0.0 : a;
            ex[j] = exponent_of(half_warp_max(a));
            code[j] = code_of(ldexp(y0, -ex[j])) | code_of(ldexp(y1, -ex[j])) << 4;
        }
    }
    const uint32_t rope = [&] {
        const float2 v = y[8];
        return pack_rn_bf16x2(v.x * c - v.y * s, v.x * s + v.y * c);
    }();
    if (write) {
        uint8_t *e = p.cache + slot * kEntry4Bytes;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            e[lane + 32 * j] = (uint8_t)code[j];
            if ((lane & 15) == 0)
                e[kScale4Offset + 2 * j + (lane >> 4)] = (uint8_t)(ex[j] + 127);
        }
        *reinterpret_cast<uint32_t *>(e + kRope4Offset + 4 * lane) = rope;
    }
    if (p.k_out) {
        uint32_t *o = p.k_out + t * p.k_out_stride;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            o[lane + 32 * j] = pack_rn_bf16x2(ldexpf(value_of(code[j] & 15u), ex[j]), ldexpf(value_of(code[j] >> 4), ex[j]));
        o[lane + 256] = rope;
    }
}

}  // namespace

cudaError_t launch_qk_norm_rope_kv_insert_fp4(const Insert4Params &p, cudaStream_t stream)
{
    if (p.num_tokens <= 0)
        return cudaSuccess;
    qk_norm_rope_kv_insert_fp4_kernel<<<p.num_tokens, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace dsv4
