// key_weights.cu -- the attention weight that a decode step gave each key, added up per cache row and position, on the
// tensor cores (tcgen05 / TMEM).
//
//   weights[row][p] += sum_h e^{scale q_h . k_p - lse_h}     for the keys p of each token's list
// with the lse that the decode returned (its sink counts there).  The lse makes the keys independent of one another: no
// maximum, no rescaling, and nothing to join where several CTAs share a token.
//
// Contraction.  S[128 keys x H heads] = K_tile[128 x 576] . Q^T, keys on the M side, so that a key's logits lie in one lane of
// tensor memory and its sum over the heads is a thread's own loop.  Q of a token (H x 576 in BF16, up to 144 KB) stays in
// shared memory; the keys come through a ring of 16-KB stages, one 64-dim column chunk of 128 keys each, dequantised to
// BF16 on the way (exactly).
//
// Roles (21 warps): warp 0 issues the products, a chunk's four as it comes; warps 1-4 read a finished block out of one of two
// accumulators, a quadrant each, while the next block is computed; warps 5-20 bring Q and the keys: two groups of eight
// take the even and the odd chunks (the rope chunk in turn), a thread half a row of a chunk, whose bytes it loaded a block
// ahead.  A persistent CTA per multiprocessor takes an equal run of the blocks of all tokens.
//
// Tokens of one row are added in ascending order, one rounding each, so the result does not depend on timing: a token
// whose row no other token of the call names is added by the epilogue, the others by a second kernel.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>

#include "serving.h"
#include "tcgen05.cuh"

namespace dsv4 {
namespace {

using namespace tc;

constexpr int kEpilogueWarps = 4;        // warps 1-4
constexpr int kKeyWarp0 = 5;
constexpr int kKeyWarps = 16;            // warps 5-20, in two groups
constexpr int kThreads = 32 * (kKeyWarp0 + kKeyWarps);
constexpr int kBK = 128;                 // keys per block = MMA M
constexpr int kChunks = 9;               // 576 dims / 64
constexpr int kStageBytes = kBK * 128;   // 16384
constexpr int kAddThreads = 512;
constexpr int kAddSlices = 16;

// N heads: Q takes 1152 N bytes; the stages fill what is left of 227 KB, up to a whole block
__host__ __device__ constexpr int stages_of(int heads) { return heads == 128 ? 5 : 9; }

// the small region after Q and the stages
constexpr int kOffLse = 0;               // float [128]: the token's lse in log2 units
constexpr int kOffBars = 512;            // u64: full[9], empty[9], d_full[2], d_empty[2], q
constexpr int kOffTmem = 704;            // u32
constexpr int kOffAbort = 708;           // int
constexpr int kOffStart = 712;           // int [2]: the unit at the run's start, and its first block
constexpr int kOffScan = 720;            // int [21]
constexpr int kSmallBytes = 832;

template <int kH>
constexpr int smem_bytes() { return kH * kDim * 2 + stages_of(kH) * kStageBytes + kSmallBytes + 1024; }

__device__ __forceinline__ uint4 ld16(const void *p) { return __ldca(reinterpret_cast<const uint4 *>(p)); }

// 32 E2M1 codes times 2^(se - 127) -> 32 BF16 values, exactly, into the 16-byte units u .. u + 3 (xored with x) of the row
// at shared address rb, in the order e0 e4 e1 e5 e2 e6 e3 e7 of each eight (a code and the one four after it lie 16 bits
// apart, so one shift puts both at their places in a BF16 pair).  A code's exponent and mantissa bits at the low end of
// the BF16 exponent are its value times 2^-126; one multiply by 2^(se - 1) gives the value.  Scales past 2 (se > 128,
// whose factor has no BF16 form) take a second multiply, 255 (NaN) among them.
__device__ __forceinline__ void store32_e2m1(const uint4 &v, uint32_t se, uint32_t rb, uint32_t u, uint32_t x)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t f = (min(se, 128u) + 126u) << 7;
    f |= f << 16;
    uint32_t g = se == 255u ? 0x7FC0u : (se - 1u) << 7;   // 2^(se - 128), where se > 128
    g |= g << 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t h = w[i] >> 8;
        uint32_t o[4] = {((w[i] << 6) & 0x01C001C0u) | ((w[i] << 12) & 0x80008000u),
                         ((w[i] << 2) & 0x01C001C0u) | ((w[i] << 8) & 0x80008000u),
                         ((h << 6) & 0x01C001C0u) | ((w[i] << 4) & 0x80008000u),
                         ((h << 2) & 0x01C001C0u) | (w[i] & 0x80008000u)};
#pragma unroll
        for (int k = 0; k < 4; ++k)
            o[k] = mul_bf16x2(o[k], f);
        if (se > 128u) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                o[k] = mul_bf16x2(o[k], g);
        }
        st_shared_v4(rb + (((u + i) ^ x) << 4), o[0], o[1], o[2], o[3]);
    }
}

// two E4M3 codes times a scale -> a BF16 pair (exact for every code and scale; NaN codes stay NaN)
__device__ __forceinline__ uint32_t convert2_e4m3(uint32_t two, float scale)
{
    const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(two & 0xFFFFu), __NV_E4M3);
    const float2 f = __half22float2(__half2(hr));
    return pack_bf16x2(f.x * scale, f.y * scale);
}

// the form of store16_e4m3 for pieces with the NaN code or a scale past 2^7, out of line
static __device__ __noinline__ void store16_e4m3_convert(uint4 v, uint32_t se, uint32_t a0, uint32_t a1)
{
    const float sc = se == 255u ? __int_as_float(0x7FC00000) : se == 0u ? __int_as_float(0x00400000) : __int_as_float((int)(se << 23));
    st_shared_v4(a0, convert2_e4m3(v.x, sc), convert2_e4m3(v.x >> 16, sc), convert2_e4m3(v.y, sc), convert2_e4m3(v.y >> 16, sc));
    st_shared_v4(a1, convert2_e4m3(v.z, sc), convert2_e4m3(v.z >> 16, sc), convert2_e4m3(v.w, sc), convert2_e4m3(v.w >> 16, sc));
}

// 16 E4M3 codes times 2^(se - 127) -> 16 BF16, elements 0-7 to shared address a0 and 8-15 to a1.  A code s.eeee.mmm placed
// as the BF16 pattern s.0000eeee.mmm0000 is its value times 2^-120; one multiply by 2^(se - 7) gives the value.
__device__ __forceinline__ void store16_e4m3(const uint4 &v, uint32_t se, uint32_t a0, uint32_t a1)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t odd = se > 134u ? 1u : 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        odd |= ((w[i] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;   // a byte with magnitude 0x7F
    if (odd != 0u) {
        store16_e4m3_convert(v, se, a0, a1);
        return;
    }
    uint32_t f = (se + 120u) << 7, o[8];
    f |= f << 16;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t t = __byte_perm(w[i >> 1], 0u, i & 1 ? 0x3424 : 0x1404);   // [0, c, 0, c']
        o[i] = mul_bf16x2((t & 0x80008000u) | ((t & 0x7F007F00u) >> 4), f);
    }
    st_shared_v4(a0, o[0], o[1], o[2], o[3]);
    st_shared_v4(a1, o[4], o[5], o[6], o[7]);
}

__device__ __forceinline__ int blocks_of(int len) { return (len + kBK - 1) / kBK; }

// The blocks of this CTA: [w, w1) of all tokens' blocks, in the order of the tokens.  Every role walks the same ones.
struct Walk {
    int w, w1;        // still to do
    int t, start;     // token of block w, and that token's first block
};

struct Segment {
    int t, len;       // token, and its keys
    int kb, nb;       // blocks kb .. kb + nb - 1 of it
};

__device__ __forceinline__ bool next_segment(Walk &k, const KeyWeightsParams &p, Segment &s)
{
    if (k.w >= k.w1)
        return false;
    while (true) {    // (tokens without keys have no block)
        s.len = __ldcg(p.lens + k.t);
        const int n = blocks_of(s.len);
        if (k.start + n > k.w) {
            s.t = k.t;
            s.kb = k.w - k.start;
            s.nb = min(n - s.kb, k.w1 - k.w);
            k.w += s.nb;
            return true;
        }
        k.start += n;
        ++k.t;
    }
}

template <int kH, bool kFour>
__global__ void __launch_bounds__(kThreads, 1) key_weights_kernel(const KeyWeightsParams p)
{
    extern __shared__ uint8_t smem_raw[];
    constexpr int kStages = stages_of(kH);
    constexpr int kQChunkBytes = kH * 128;
    constexpr uint32_t kTmemCols = kH < 16 ? 32 : 2 * kH;
    // instruction descriptor (kind::f16): D f32, A/B bf16, both K-major
    constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(kH >> 3) << 17) | ((uint32_t)(kBK >> 4) << 24);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;   // the swizzled tiles start on 1024-byte boundaries
    const uint32_t sQ = base, sK = base + kChunks * kQChunkBytes;
    uint8_t *small = smem_raw + (base - raw) + kChunks * kQChunkBytes + kStages * kStageBytes;
    float *slse = reinterpret_cast<float *>(small + kOffLse);
    const uint32_t bar_full = smem_u32(small + kOffBars);      // [stage] written (a group's eight warps)
    const uint32_t bar_empty = bar_full + 8 * 9;               // [stage] read by its products
    const uint32_t bar_dfull = bar_full + 8 * 18;              // [2] the block's products are complete
    const uint32_t bar_dempty = bar_full + 8 * 20;             // [2] read by the epilogue
    const uint32_t bar_q = bar_full + 8 * 22;                  // Q of the segment written
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(small + kOffTmem);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(small + kOffAbort);
    int *first = reinterpret_cast<int *>(small + kOffStart);
    int *scan = reinterpret_cast<int *>(small + kOffScan);

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(bar_full + 8 * i, kKeyWarps / 2);
            mbar_init(bar_empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar_dfull + 8 * i, 1);
            mbar_init(bar_dempty + 8 * i, kEpilogueWarps);
        }
        mbar_init(bar_q, kKeyWarps);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        *abort_flag = 0;
    }
    // (only the list kernel can still be running ahead of this one: it waited for what came before)
    if (warp == 0)
        tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    griddep_wait();

    // ---- this CTA's blocks
    Walk walk;
    {
        const int per = (p.num_tokens + kThreads - 1) / kThreads;
        const int t0 = min(p.num_tokens, tid * per), t1 = min(p.num_tokens, t0 + per);
        int mine = 0;
        for (int t = t0; t < t1; ++t)
            mine += blocks_of(__ldcg(p.lens + t));
        int incl = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d)
                incl += y;
        }
        if (lane == 31)
            scan[warp] = incl;
        __syncthreads();
        int at = incl - mine, W = 0;
        for (int i = 0; i < kThreads / 32; ++i) {
            at += i < warp ? scan[i] : 0;
            W += scan[i];
        }
        walk.w = (int)((long long)W * blockIdx.x / gridDim.x);
        walk.w1 = (int)((long long)W * (blockIdx.x + 1) / gridDim.x);
        if (walk.w < walk.w1 && mine > 0 && at <= walk.w && walk.w < at + mine) {
            int t = t0, n;
            while (at + (n = blocks_of(__ldcg(p.lens + t))) <= walk.w) {
                at += n;
                ++t;
            }
            first[0] = t;
            first[1] = at;
        }
        before_sync();
        __syncthreads();
        after_sync();
        walk.t = first[0];
        walk.start = first[1];
    }
    const uint32_t tmem = *tmem_slot;
    griddep_launch();   // (the adding kernel waits for this grid itself)
    Segment seg;
    uint32_t g = 0;     // blocks since the kernel began

    if (warp == 0) {
        // ---- the products: K-major operands advance 32 B per 16 dims and one chunk per 64
        const uint32_t leader = elect_one();
        const uint64_t da = sdesc(sK, 16, 1024), db = sdesc(sQ, 16, 1024);
        uint32_t stage = 0, phase = 0;
        for (uint32_t n = 0; next_segment(walk, p, seg); ++n) {
            mbar_wait(bar_q, n & 1u, abort_flag, p.status);
            for (int b = 0; b < seg.nb; ++b, ++g) {
                const uint32_t x = g & 1u;
                if (g >= 2) {
                    mbar_wait(bar_dempty + 8 * x, ((g >> 1) - 1) & 1u, abort_flag, p.status);
                    after_sync();
                }
#pragma unroll 1
                for (int c = 0; c < kChunks; ++c) {
                    mbar_wait(bar_full + 8 * stage, phase, abort_flag, p.status);
                    after_sync();
                    const uint64_t a = da + (uint64_t)((stage * kStageBytes) >> 4), bq = db + (uint64_t)((c * kQChunkBytes) >> 4);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_bf16(leader, tmem + kH * x, a + (uint64_t)(2 * k), bq + (uint64_t)(2 * k), kIdesc, (c != 0 || k != 0) ? 1u : 0u);
                    commit(leader, bar_empty + 8 * stage);
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                commit(leader, bar_dfull + 8 * x);
            }
        }
    } else if (warp < kKeyWarp0) {
        // ---- sums over the heads: lane l of quadrant q has key 32 q + l of the block
        const int quad = warp & 3, row = 32 * quad + lane;
        const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
        const float c2 = p.scale * 1.4426950408889634f;
        while (next_segment(walk, p, seg)) {
            const int t = seg.t;
            const int r = p.req_idx != nullptr ? __ldcg(p.req_idx + t) : t;
            const bool sole = __ldcg(p.sole + t) != 0;
            named_bar(1, 32 * kEpilogueWarps);   // (slse has been read)
            if (row < kH) {
                const float l = __ldcg(p.lse + (int64_t)t * kH + row);
                slse[row] = l == -INFINITY ? -INFINITY : l * -1.4426950408889634f;   // (a head without weight)
            }
            named_bar(1, 32 * kEpilogueWarps);
            for (int b = 0; b < seg.nb; ++b, ++g) {
                const uint32_t x = g & 1u;
                const int i = (seg.kb + b) * kBK + row;
                const int64_t at = (int64_t)t * p.list_w + i;
                float *place = nullptr;
                float had = 0.f;
                if (i < seg.len && __ldcg(p.slots + at) >= 0) {
                    place = sole ? p.weights + (int64_t)r * p.weights_stride + __ldcg(p.positions + at) : p.got + at;
                    if (sole)
                        had = __ldcg(place);
                }
                mbar_wait(bar_dfull + 8 * x, (g >> 1) & 1u, abort_flag, p.status);
                after_sync();
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int h = 0; h < kH; h += 16) {
                    uint32_t s[16];
                    tmem_ld16(lane_base + kH * x + h, s);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        const float4 l = *reinterpret_cast<const float4 *>(slse + h + j);
                        sum[0] += exp2_approx(fmaf(__uint_as_float(s[j]), c2, l.x));
                        sum[1] += exp2_approx(fmaf(__uint_as_float(s[j + 1]), c2, l.y));
                        sum[2] += exp2_approx(fmaf(__uint_as_float(s[j + 2]), c2, l.z));
                        sum[3] += exp2_approx(fmaf(__uint_as_float(s[j + 3]), c2, l.w));
                    }
                }
                before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar_dempty + 8 * x);
                if (place != nullptr)
                    __stcg(place, had + ((sum[0] + sum[1]) + (sum[2] + sum[3])));
            }
        }
    } else {
        // ---- Q and the keys.  A thread has dims [32 half, 32 half + 32) of row `row` of its group's chunks
        const int kw = warp - kKeyWarp0, group = kw >> 3, gid = 32 * (kw & 7) + lane;
        const int row = gid >> 1, half = gid & 1;
        const uint32_t rb = (uint32_t)(row >> 3) * 1024u + (uint32_t)(row & 7) * 128u, x7 = (uint32_t)(row & 7);
        constexpr int kPieces = kFour ? 1 : 2;           // 16-byte pieces of 32 values
        for (uint32_t n = 0; next_segment(walk, p, seg); ++n) {
            const int t = seg.t;
            const int32_t *list = p.slots + (int64_t)t * p.list_w;
            auto load_slot = [&](int b) {
                const int i = (seg.kb + b) * kBK + row;
                return b < seg.nb && i < seg.len ? __ldcg(list + i) : -1;
            };
            auto entry_of = [&](int slot) { return p.kv + (int64_t)max(slot, 0) * (kFour ? kEntry4Bytes : kEntryBytes); };
            // the entry of the block ahead: pieces of chunks group, group + 2, ..; rope in the blocks of this group's turn
            uint4 pre[4][kPieces], rope[4], scales;
            auto load_piece = [&](const uint8_t *e, int i) {
                const int chunk = group + 2 * i;
#pragma unroll
                for (int k = 0; k < kPieces; ++k)
                    pre[i][k] = ld16(e + (kFour ? 32 * chunk + 16 * half : 64 * chunk + 32 * half + 16 * k));
            };
            auto load_scales = [&](const uint8_t *e) {
                if (kFour)
                    scales = ld16(e + kScale4Offset);
                else
                    scales.x = __ldca(reinterpret_cast<const uint32_t *>(e + kScaleOffset));
            };
            auto load_rope = [&](const uint8_t *e) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    rope[i] = ld16(e + (kFour ? kRope4Offset : kRopeOffset) + 64 * half + 16 * i);
            };
            int slot = load_slot(0), slot_next = load_slot(1);
            if (slot >= 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    load_piece(entry_of(slot), i);
                load_scales(entry_of(slot));
                if ((int)(g & 1u) == group)
                    load_rope(entry_of(slot));
            }
            if (n > 0)   // the products of the last segment are done with its Q
                mbar_wait(bar_dfull + 8 * ((g - 1) & 1u), ((g - 1) >> 1) & 1u, abort_flag, p.status);
            {
                const uint4 *q = reinterpret_cast<const uint4 *>(p.q + (int64_t)t * p.q_token_stride);
                constexpr int kLoads = (kH * (kDim / 8) + 32 * kKeyWarps - 1) / (32 * kKeyWarps);
                constexpr int kBatch = kLoads < 6 ? kLoads : 6;
#pragma unroll 1
                for (int j0 = 0; j0 < kLoads; j0 += kBatch) {
                    uint4 v[kBatch];
#pragma unroll
                    for (int j = 0; j < kBatch; ++j) {
                        const int i = 32 * kKeyWarps * (j0 + j) + 32 * kw + lane;
                        if (i < kH * (kDim / 8))
                            v[j] = __ldca(q + i);
                    }
#pragma unroll
                    for (int j = 0; j < kBatch; ++j) {
                        const int i = 32 * kKeyWarps * (j0 + j) + 32 * kw + lane;
                        if (i >= kH * (kDim / 8))
                            break;
                        const int h = i / (kDim / 8), c = i % (kDim / 8);
                        const uint32_t a = sQ + (c >> 3) * kQChunkBytes + sw128(h, c & 7);
                        if (kFour && c < kLatent / 8)   // (the order of the latent dims that store32_e2m1 gives)
                            st_shared_v4(a, __byte_perm(v[j].x, v[j].z, 0x5410), __byte_perm(v[j].x, v[j].z, 0x7632),
                                         __byte_perm(v[j].y, v[j].w, 0x5410), __byte_perm(v[j].y, v[j].w, 0x7632));
                        else
                            st_shared_v4(a, v[j].x, v[j].y, v[j].z, v[j].w);
                    }
                }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar_q);

            for (int b = 0; b < seg.nb; ++b, ++g) {
                const bool ok = slot >= 0, ok_next = slot_next >= 0;
                const uint8_t *next = entry_of(slot_next);
                const uint4 sc = scales;
                if (ok_next)
                    load_scales(next);
                // a stage for chunk c: wait until its last products are complete, and then tell that it is written
                auto begin = [&](int c) {
                    const uint32_t at = g * kChunks + c, stage = at % kStages;
                    if (at >= kStages)
                        mbar_wait(bar_empty + 8 * stage, ((at / kStages) & 1u) ^ 1u, abort_flag, p.status);
                    return stage;
                };
                auto end = [&](uint32_t stage) {
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(bar_full + 8 * stage);
                };
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t stage = begin(group + 2 * i);
                    const uint32_t a = sK + stage * kStageBytes + rb;
                    if (!ok) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            st_shared_v4(a + (((4 * half + k) ^ x7) << 4), 0u, 0u, 0u, 0u);
                    } else if (kFour) {
                        const uint32_t word = i == 0 ? sc.x : i == 1 ? sc.y : i == 2 ? sc.z : sc.w;
                        store32_e2m1(pre[i][0], (word >> (8 * (2 * group + half))) & 255u, a, 4 * half, x7);
                    } else {
                        const uint32_t se = (sc.x >> (8 * i)) & 255u;
#pragma unroll
                        for (int k = 0; k < kPieces; ++k)
                            store16_e4m3(pre[i][k], se, a + (((4 * half + 2 * k) ^ x7) << 4), a + (((4 * half + 2 * k + 1) ^ x7) << 4));
                    }
                    if (ok_next)
                        load_piece(next, i);
                    end(stage);
                }
                if ((int)(g & 1u) == group) {
                    const uint32_t stage = begin(8);
                    const uint32_t a = sK + stage * kStageBytes + rb;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint4 v = ok ? rope[i] : make_uint4(0u, 0u, 0u, 0u);
                        st_shared_v4(a + (((4 * half + i) ^ x7) << 4), v.x, v.y, v.z, v.w);
                    }
                    end(stage);
                } else if (ok_next) {
                    load_rope(next);
                }
                slot = slot_next;
                slot_next = load_slot(b + 2);
            }
        }
    }
    before_sync();
    __syncthreads();
    after_sync();
    if (warp == 0)
        tmem_free(tmem, kTmemCols);
}

// Tokens that share a row, one after the other; positions are dealt out to the slices in runs of 256.
__global__ void __launch_bounds__(kAddThreads) add_weights_kernel(const KeyWeightsParams p)
{
    griddep_wait();
    griddep_launch();
    const int r = blockIdx.y, slice = blockIdx.x, tid = threadIdx.x;
    float *row = p.weights + (int64_t)r * p.weights_stride;
    for (int t = 0; t < p.num_tokens; ++t) {
        if (p.req_idx[t] != r || __ldcg(p.sole + t) != 0)
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

template <int kH, bool kFour>
cudaError_t launch(const KeyWeightsParams &p, int sms, cudaStream_t stream)
{
    const auto kernel = key_weights_kernel<kH, kFour>;
    constexpr int kSlot = kAttrKeyWeights + (kH == 16 ? 0 : kH == 32 ? 1 : kH == 64 ? 2 : 3) + (kFour ? 4 : 0);
    const cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kernel), smem_bytes<kH>(), (AttrSlot)kSlot);
    if (e != cudaSuccess)
        return e;
    return launch_dependent(kernel, dim3((unsigned)sms), kThreads, smem_bytes<kH>(), stream, p);
}

template <bool kFour>
cudaError_t launch_for(const KeyWeightsParams &p, int sms, cudaStream_t stream)
{
    switch (p.num_heads) {
    case 16: return launch<16, kFour>(p, sms, stream);
    case 32: return launch<32, kFour>(p, sms, stream);
    case 64: return launch<64, kFour>(p, sms, stream);
    case 128: return launch<128, kFour>(p, sms, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace

int key_weights_block_keys() { return kBK; }

cudaError_t launch_key_weights(const KeyWeightsParams &p, int sms, cudaStream_t stream)
{
    const cudaError_t e = p.entry_bytes == kEntry4Bytes ? launch_for<true>(p, sms, stream) : launch_for<false>(p, sms, stream);
    if (e != cudaSuccess || p.req_idx == nullptr)   // (without req_idx every token has a row of its own)
        return e;
    return launch_dependent(add_weights_kernel, dim3(kAddSlices, (unsigned)p.num_reqs), kAddThreads, 0, stream, p);
}

}  // namespace dsv4
