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
// Work.  A warp per four heads of a token, a warp per key.  Eight lanes share a head, each with nine 16-byte pieces
// (8 values) of its 1152 bytes, so a load or store covers 128 contiguous bytes of four heads, the sum of squares takes
// three shuffles for all four, and no lane is idle; all loads of a warp are in flight before any use.  Bound by HBM:
// every query is read and written once.  (Pairs of 4 bytes to a lane and a warp to a head took 2.4 times as long for
// 8191 tokens x 64 heads; queries whose rows are not 16-byte aligned still go by fours of such loads.)  The keys' warps
// come first: their fp64 chain is the longest.
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

// four pairs at a (16-byte aligned when kWide)
template <bool kWide>
__device__ __forceinline__ uint4 load4(const uint32_t *a)
{
    if (kWide)
        return __ldg(reinterpret_cast<const uint4 *>(a));
    return make_uint4(__ldg(a), __ldg(a + 1), __ldg(a + 2), __ldg(a + 3));
}

template <bool kWide>
__device__ __forceinline__ void store4(uint32_t *a, const uint32_t (&v)[4])
{
    if (kWide) {
        *reinterpret_cast<uint4 *>(a) = make_uint4(v[0], v[1], v[2], v[3]);
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
        c = make_float4(__ldg(cs), __ldg(cs + 1), __ldg(cs + 2), __ldg(cs + 3));
        s = make_float4(__ldg(cs + 32), __ldg(cs + 33), __ldg(cs + 34), __ldg(cs + 35));
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
        const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
        uint32_t y[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 v = unpack_bf16x2(w[k]);
            float y0 = v.x * r, y1 = v.y * r;
            if (p.q_w != nullptr) {
                const float2 g = make_float2(__ldg(p.q_w + 64 * j + 8 * l8 + 2 * k), __ldg(p.q_w + 64 * j + 8 * l8 + 2 * k + 1));
                y0 *= g.x;
                y1 *= g.y;
            }
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
        c = __ldg(p.cos_sin + pos * 64 + lane);
        s = __ldg(p.cos_sin + pos * 64 + 32 + lane);
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

// kWide: the queries' rows are 16-byte aligned
template <bool kWide>
__global__ void __launch_bounds__(kThreads, 3) qk_norm_rope_kv_insert_fp4_kernel(const Insert4Params p)
{
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
    const bool wide = (((reinterpret_cast<uintptr_t>(p.q) | reinterpret_cast<uintptr_t>(p.q_out)) & 15u) == 0) &&
                      ((p.q_stride | p.q_out_stride) & 3) == 0;
    if (wide)
        qk_norm_rope_kv_insert_fp4_kernel<true><<<(unsigned)grid, kThreads, 0, stream>>>(p);
    else
        qk_norm_rope_kv_insert_fp4_kernel<false><<<(unsigned)grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace dsv4
