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
// rounding border would be off by all of it.  The key is computed in fp32 too, with a check whether any value of a
// block, or its maximum, lies so near to a border that roundings could decide (kNear); the pairs of blocks that have one
// (about one in 3500 of normal keys) are done again in fp64.
//
// Work.  A warp per four heads of a token, a warp per key.  Eight lanes share a head, each with nine 16-byte pieces
// (8 values) of its 1152 bytes, so a load or store covers 128 contiguous bytes of four heads, the sum of squares takes
// three shuffles for all four, and no lane is idle; all loads of a warp are in flight before any use.  Bound by HBM:
// every query is read and written once (8191 tokens x 64 heads: 183 us, 1.23 GB, the rate of a copy; 128 x 128: 7.4 us).
// (Pairs of 4 bytes to a lane and a warp to a head took 477 us; queries whose rows are not 16-byte aligned still go by
// fours of such loads.)  The keys' warps come first: their fp64 chain is the longest.
#include <climits>
#include <cuda_bf16.h>
#include <cuda_fp4.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fp4.h"

namespace dsv4 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPairs = kDim / 2;   // 288 BF16 pairs per head; pairs 256.. are the rope part
// What a key's value may be off by in fp32, in roundings of 2^-24 of it.  Over 576 dims: the sum of squares 17 to a lane (of
// 18 products the first is exact) and 5 levels, the mean 1, eps 1, adding it 1: 25, halved by the root; the root, its
// reciprocal and two products 4: 16.5.  (512 dims: 15 by the same count, dividing by them is exact.)  The comparison's own
// product rounds once more: 17.5 in all, below 20.  (The window of exponent_of: 16 steps of 2^-23 at 1.5, 21 roundings.)
constexpr float kNear = 0x1.4p-20f;

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

template <typename T>
__device__ __forceinline__ T warp_sum(T v)
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

// Smallest integer e with 6 * 2^e >= amax (0 for amax 0), clamped to [-127, 125]: k - 2 for amax in [2^k, 1.5 * 2^k],
// k - 1 from there to 2^(k+1).  *near: amax is within 21 roundings of the border 1.5 * 2^k, or too small to tell.
__device__ __forceinline__ int exponent_of(float amax, bool *near)
{
    const int bits = __float_as_int(amax), m = bits & 0x7FFFFF;
    *near = (unsigned)(m - 0x400000 + 16) <= 32u || (amax < 0x1p-100f && amax > 0.f);
    if (bits == 0)
        return 0;
    return max(-127, min(125, (bits >> 23) - 129 + (m > 0x400000 ? 1 : 0)));
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

// the value of a code times 2^e (a code's bits at the low end of an fp32 exponent are its value times 2^-126)
__device__ __forceinline__ float value_of(uint32_t code, int e)
{
    const float m = __uint_as_float(((code & 7u) << 22) | ((code & 8u) << 28)) * 0x1p126f;
    return e < -126 ? m * 0x1p-126f * 0.5f : m * pow2f(e);
}

// Block pair j of token t's key (values of pairs lane + 32 j) in fp64: the lane's two codes, and its half warp's block
// exponent + 127 from bit 8.
__device__ __noinline__ uint32_t exact_codes(const Insert4Params &p, int t, int j, int lane)
{
    const uint32_t *a = p.kv + t * p.kv_stride + lane;
    const int nj = p.kv_norm_dims / 64;
    double ss = 0.0;
    for (int i = 0; i < nj; ++i) {
        const float2 v = unpack_bf16x2(__ldca(a + 32 * i));
        ss = fma((double)v.x, (double)v.x, fma((double)v.y, (double)v.y, ss));
    }
    const double root = sqrt(warp_sum(ss) / (double)p.kv_norm_dims + p.eps);
    const float2 v = unpack_bf16x2(__ldca(a + 32 * j));
    const int d = 2 * (lane + 32 * j);
    const double y0 = (double)v.x / root * (p.kv_w ? (double)__ldca(p.kv_w + d) : 1.0);
    const double y1 = (double)v.y / root * (p.kv_w ? (double)__ldca(p.kv_w + d + 1) : 1.0);
    const double a0 = isnan(y0) ? 0.0 : fabs(y0), a1 = isnan(y1) ? 0.0 : fabs(y1);
    const int e = exponent_of(half_warp_max(a0 > a1 ? a0 : a1));
    return code_of(ldexp(y0, -e)) | code_of(ldexp(y1, -e)) << 4 | (uint32_t)(e + 127) << 8;
}

// 16 bytes at a (16-byte aligned when kWide)
template <bool kWide>
__device__ __forceinline__ uint4 load4(const void *a)
{
    if (kWide)
        return __ldca(reinterpret_cast<const uint4 *>(a));
    const uint32_t *b = static_cast<const uint32_t *>(a);
    return make_uint4(__ldca(b), __ldca(b + 1), __ldca(b + 2), __ldca(b + 3));
}

__device__ __forceinline__ float4 as_floats(const uint4 &v)
{
    return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
}

// The queries stream through: written so that they leave L2 first, they do not push out what else the step keeps
// there (128 tokens x 128 heads: 7.4 against 11.4 us with the inputs of other calls in L2; 8191 x 64: the same).
template <bool kWide>
__device__ __forceinline__ void store4(uint32_t *a, const uint32_t (&v)[4])
{
    if (kWide) {
        __stcs(reinterpret_cast<uint4 *>(a), make_uint4(v[0], v[1], v[2], v[3]));
    } else {
        a[0] = v[0];
        a[1] = v[1];
        a[2] = v[2];
        a[3] = v[3];
    }
}

// Heads 4 quad .. 4 quad + 3 of token t.
template <bool kWide>
__device__ __forceinline__ void norm_rope_queries(const Insert4Params &p, int t, int quad, int lane)
{
    const int h = 4 * quad + (lane >> 3), l8 = lane & 7;
    const bool there = h < p.num_heads;
    const int64_t pos = p.positions[t];
    const uint32_t *a = p.q + t * p.q_stride + (int64_t)(there ? h : 4 * quad) * kPairs + 4 * l8;
    uint4 x[9];   // pieces l8 + 8 j of the head; j = 8: rope pairs 4 l8 .. 4 l8 + 3
#pragma unroll
    for (int j = 0; j < 9; ++j)
        x[j] = load4<kWide>(a + 32 * j);
    const bool rot = pos >= 0 && pos < p.max_pos;
    float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (rot) {
        const float *cs = p.cos_sin + pos * 64 + 4 * l8;
        c = as_floats(load4<kWide>(cs));
        s = as_floats(load4<kWide>(cs + 32));
    }
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < 9; ++j) {
        const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 v = unpack_bf16x2(w[k]);
            ss = fmaf(v.x, v.x, fmaf(v.y, v.y, ss));
        }
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1)
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = 1.f / sqrtf(ss / (float)kDim + (float)p.eps);
    uint32_t *o = p.q_out + t * p.q_out_stride + (int64_t)h * kPairs + 4 * l8;
#pragma unroll
    for (int j = 0; j < 9; ++j) {
        // (kept packed across the reduction: unpacked, the 72 values of a lane would spill)
        asm volatile("" : "+r"(x[j].x), "+r"(x[j].y), "+r"(x[j].z), "+r"(x[j].w));
        const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
        float4 g[2] = {make_float4(1.f, 1.f, 1.f, 1.f), make_float4(1.f, 1.f, 1.f, 1.f)};
        if (p.q_w != nullptr) {
            g[0] = as_floats(load4<kWide>(p.q_w + 64 * j + 8 * l8));
            g[1] = as_floats(load4<kWide>(p.q_w + 64 * j + 8 * l8 + 4));
        }
        uint32_t y[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 v = unpack_bf16x2(w[k]);
            float y0 = v.x * r * (k & 1 ? g[k >> 1].z : g[k >> 1].x), y1 = v.y * r * (k & 1 ? g[k >> 1].w : g[k >> 1].y);
            if (j == 8) {
                const float ck = k == 0 ? c.x : k == 1 ? c.y : k == 2 ? c.z : c.w;
                const float sk = k == 0 ? s.x : k == 1 ? s.y : k == 2 ? s.z : s.w;
                const float u = y0 * ck - y1 * sk;
                y1 = y0 * sk + y1 * ck;
                y0 = u;
            }
            y[k] = pack_rn_bf16x2(y0, y1);
        }
        if (there)
            store4<kWide>(o + 32 * j, y);
    }
}

// Token t's key.  Lane l holds the BF16 pairs l + 32 j (j < 9; j = 8 is the rope part, pair i = l), so half a warp holds
// a block of 32 values.
__device__ __forceinline__ void insert_key(const Insert4Params &p, int t, int lane)
{
    const int64_t pos = p.positions[t];
    const bool rot = pos >= 0 && pos < p.max_pos;
    float c = 1.f, s = 0.f;   // this lane's rope pair i = lane
    if (rot) {
        c = __ldca(p.cos_sin + pos * 64 + lane);
        s = __ldca(p.cos_sin + pos * 64 + 32 + lane);
    } else if (lane == 0) {
        atomicOr(p.status, kStatusBadIndex);
    }
    const int64_t slot = p.slots[t];
    if (lane == 0 && slot >= p.num_slots)
        atomicOr(p.status, kStatusBadIndex);
    const bool write = slot >= 0 && slot < p.num_slots && rot;
    uint32_t x[9];
#pragma unroll
    for (int j = 0; j < 9; ++j)
        x[j] = __ldca(p.kv + t * p.kv_stride + lane + 32 * j);
    const int nj = p.kv_norm_dims / 64;   // pairs lane + 32 j with j < nj are normalised
    float r = 1.f;
    if (nj > 0) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 9; ++j) {
            const float2 v = unpack_bf16x2(x[j]);
            if (j < nj)
                ss = fmaf(v.x, v.x, fmaf(v.y, v.y, ss));
        }
        r = 1.f / sqrtf(warp_sum(ss) / (float)p.kv_norm_dims + (float)p.eps);
    }
    // the sum of squares of such keys may pass fp32's range (or the root lose its precision): all in fp64
    const bool wild = nj > 0 && !(r > 0x1p-60f && r < 0x1p60f);
    uint8_t *e = p.cache + (write ? slot : 0) * kEntry4Bytes;
    uint32_t *o = p.k_out + t * p.k_out_stride;
#pragma unroll
    for (int j = 0; j < 8; ++j) {   // blocks 2 j (lanes 0..15) and 2 j + 1 (lanes 16..31)
        const float2 v = unpack_bf16x2(x[j]);
        float y0 = v.x, y1 = v.y;
        if (j < nj) {
            y0 *= r;
            y1 *= r;
            if (p.kv_w != nullptr) {
                y0 *= __ldca(p.kv_w + 2 * (lane + 32 * j));
                y1 *= __ldca(p.kv_w + 2 * (lane + 32 * j) + 1);
            }
        }
        bool near;
        int ex = exponent_of(half_warp_max(fmaxf(fmaxf(fabsf(y0), fabsf(y1)), 0.f)), &near);   // (a NaN counts as 0)
        const float f = pow2f(-ex), t0 = y0 * f, t1 = y1 * f;
        uint32_t code = codes_of(t0, t1);
        if (nj > 0) {   // (without a norm the key is BF16 and everything above is exact)
            near |= wild || codes_of(t0 * (1.f - kNear), t1 * (1.f - kNear)) != codes_of(t0 * (1.f + kNear), t1 * (1.f + kNear));
            if (__any_sync(0xffffffffu, near)) {
                const uint32_t c = exact_codes(p, t, j, lane);
                code = c & 0xFFu;
                ex = (int)(c >> 8) - 127;
            }
        }
        if (write) {
            e[lane + 32 * j] = (uint8_t)code;
            if ((lane & 15) == 0)
                e[kScale4Offset + 2 * j + (lane >> 4)] = (uint8_t)(ex + 127);
        }
        if (p.k_out != nullptr)
            o[lane + 32 * j] = pack_rn_bf16x2(value_of(code & 15u, ex), value_of(code >> 4, ex));
    }
    float2 v = unpack_bf16x2(x[8]);
    if (nj > 8) {
        v.x *= r;
        v.y *= r;
        if (wild) {   // (as the latent: from the fp64 root)
            double ss = 0.0;
            for (int i = 0; i < 9; ++i) {
                const float2 u = unpack_bf16x2(__ldca(p.kv + t * p.kv_stride + lane + 32 * i));
                ss = fma((double)u.x, (double)u.x, fma((double)u.y, (double)u.y, ss));
            }
            const double root = sqrt(warp_sum(ss) / (double)kDim + p.eps);
            const float2 u = unpack_bf16x2(x[8]);
            v = make_float2((float)((double)u.x / root), (float)((double)u.y / root));
        }
        if (p.kv_w != nullptr) {
            v.x *= __ldca(p.kv_w + kLatent + 2 * lane);
            v.y *= __ldca(p.kv_w + kLatent + 2 * lane + 1);
        }
    }
    const uint32_t rope = pack_rn_bf16x2(v.x * c - v.y * s, v.x * s + v.y * c);
    if (write)
        *reinterpret_cast<uint32_t *>(e + kRope4Offset + 4 * lane) = rope;
    if (p.k_out != nullptr)
        o[256 + lane] = rope;
}

// kWide: the queries' rows, their weight and the rotation table are 16-byte aligned
template <bool kWide>
__global__ void __launch_bounds__(kThreads, 4) qk_norm_rope_kv_insert_fp4_kernel(const Insert4Params p)
{
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int quads = (p.num_heads + 3) / 4;
    if (item < p.num_tokens)
        insert_key(p, (int)item, lane);
    else if (item < (int64_t)p.num_tokens * (1 + quads))
        norm_rope_queries<kWide>(p, (int)((item - p.num_tokens) / quads), (int)((item - p.num_tokens) % quads), lane);
}

}  // namespace

cudaError_t launch_qk_norm_rope_kv_insert_fp4(const Insert4Params &p, cudaStream_t stream)
{
    if (p.num_tokens <= 0)
        return cudaSuccess;
    const long long items = (long long)p.num_tokens * (1 + (p.num_heads + 3) / 4);
    const long long grid = (items + kWarps - 1) / kWarps;
    if (grid > INT_MAX)
        return cudaErrorInvalidValue;
    const bool wide = (((reinterpret_cast<uintptr_t>(p.q) | reinterpret_cast<uintptr_t>(p.q_out) |
                         reinterpret_cast<uintptr_t>(p.q_w) | reinterpret_cast<uintptr_t>(p.cos_sin)) & 15u) == 0) &&
                      ((p.q_stride | p.q_out_stride) & 3) == 0;
    return launch_dependent(wide ? qk_norm_rope_kv_insert_fp4_kernel<true> : qk_norm_rope_kv_insert_fp4_kernel<false>,
                            dim3((unsigned)grid), kThreads, 0, stream, p);
}

}  // namespace dsv4
