// key_weights.cu -- the attention weight that a decode step gave each key, added up per cache row and position, on the
// tensor cores (tcgen05 / TMEM).
//
//   weights[row][p] += sum_h e^{scale q_h . k_p - lse_h}     for the keys p of each token's list
// with the lse that the decode returned (its sink counts there).  The lse makes the keys independent of one another: no
// maximum, no rescaling, and nothing to join where several CTAs share a token.
//
// Contraction.  S[128 keys x H heads] = K_tile[128 x 576] . Q^T, keys on the M side, so that a key's logits lie in one lane of
// tensor memory and its sum over the heads is a thread's own loop.  Q of a token (H x 576 in BF16, up to 144 KB) stays in
// shared memory.  The entries come whole, by asynchronous 16-byte copies, into a ring of 16-key units for each quadrant; a thread
// takes its 64-dim chunks out of one, dequantises them to BF16 (exactly) and writes them to tensor memory, from where the
// product reads them: written to shared memory instead, the keys' stores and the products' reads of both operands (and loads to
// registers, whose pieces of 16 or 32 bytes a row take a pass of L1 each) kept L1 busy for 80 % of the time.
//
// Roles (24 warps): warp 0 issues the products; warps 1-4 read a finished block out of one of two accumulators, a quadrant
// each, while the next block is computed; warps 5 and 6 copy entries; warps 7-22 dequantise, in four sets, a warp a quadrant, and
// bring the CTA's first Q; warp 23 brings the Q of later tokens, in three groups of chunks, each as soon as the last products
// with what stood there are done.  A persistent CTA per multiprocessor takes an equal run of the blocks of all tokens.
//
// What bounds it (128 heads, 10 blocks a CTA): 54 us for 128 tokens of 8-bit entries and 35 for 6 histories of 20000 to 40000 4-bit ones, of
// which this kernel takes 28 to 36 and 26.  A CTA's first products start 4 us after it (lengths, slots, entries, Q: 200 KB
// through an L1 that takes 43 bytes a cycle); then a block takes 6.3 k cycles (8-bit) or 4.2 k, where its products are
// 2.3 k.  Copying a block takes the two warps 3.6 k cycles, dequantising it the sixteen 3.3 k, and with two to three units to a
// quadrant beside Q one waits for the other: the copies, whose rows of 400 or 656 bytes never fill L1's lines (64 bytes a row take 21
// cycles for 512 bytes, 24 bytes a cycle at most; 12 cycles where a warp's lanes are neighbours).  Slower: a third copy warp (63 / 46 us),
// 128 bytes a row (58 / 38), bulk copies for a quarter or an eighth of the rows (60 / 43; one takes its warp 60 cycles), units
// finished by one lane after a wait for the group (59 / 38).
//
// Tokens of one row are added in ascending order, one rounding each, so the result does not depend on timing: the first
// token with keys that names a row is added by the epilogue, the others by a second kernel.
#include <algorithm>
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
constexpr int kCopyWarp0 = 5;
constexpr int kCopyWarps = 2;            // warps 5 and 6, two quadrants each
constexpr int kKeyWarp0 = kCopyWarp0 + kCopyWarps;
constexpr int kKeyWarps = 16;            // warps 7-22, in four sets
constexpr int kSets = kKeyWarps / 4;
constexpr int kQWarp = kKeyWarp0 + kKeyWarps;   // warp 23
constexpr int kThreads = 32 * (kQWarp + 1);
constexpr int kBK = 128;                 // keys per block = MMA M
constexpr int kChunks = 9;               // 576 dims / 64
constexpr int kQGroups = 3;              // of Q, three chunks each in the order of the products
constexpr int kSlots = 8;                // chunks in tensor memory, 32 columns each
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColKeys = 256;       // (two accumulators of up to 128 columns before them)
constexpr int kMaxDepth = 4;             // units of a quadrant's ring
constexpr int kSwitch = 1;               // blocks' worth of time that a token's start takes (some 1 us; the dearest CTAs set the time)
constexpr int kLongRun = 4;              // blocks to a CTA from which on the starts count (with fewer, some would get none)
constexpr int kAddThreads = 256;
constexpr int kAddSlices = 4;
constexpr int kFront = 8;                // entries of a token that a thread has in flight
constexpr int kAddRows = 1 << 20;        // rows at a time

// the small region after Q and the units
constexpr int kOffLse = 0;               // float [128]: the token's lse in log2 units; before that int2 [24]: a sum over the warps
constexpr int kOffBars = 512;            // u64: raw_full[16], raw_empty[16], full[8], empty[8], d_full[2], d_empty[2],
                                         // q[3], q_free[3], q_raw[3]
constexpr int kOffTmem = 1008;           // u32
constexpr int kOffAbort = 1012;          // int
constexpr int kOffStart = 1016;          // int [2]: the token at the run's start, and its first block
constexpr int kSmallBytes = 1024;
static_assert(kOffBars + 8 * (8 * kMaxDepth + 2 * kSlots + 4 + 3 * kQGroups) <= kOffTmem && 8 * (kThreads / 32) <= kOffBars, "small region");

// N heads: Q takes 1152 N bytes; units of 16 entries fill what is left of 227 KB
template <int kH, bool kFour>
struct Shape {
    static constexpr int kEntry = kFour ? kEntry4Bytes : kEntryBytes;
    static constexpr int kUnitBytes = 16 * kEntry;
    static constexpr int kRoom = (232448 - kSmallBytes - kH * kDim * 2) / (4 * kUnitBytes);
    static constexpr int kDepth = kRoom < kMaxDepth ? kRoom : kMaxDepth;
    static constexpr int kSmem = kH * kDim * 2 + 4 * kDepth * kUnitBytes + kSmallBytes;
    // (a block's chunks are consumed in all four quadrants together, so a whole block has to fit)
    static_assert(kDepth >= 2, "units");
};

__device__ __forceinline__ uint4 lds16(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

__device__ __forceinline__ uint32_t lds8(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

// A (BF16 pairs, K along the columns) from tensor memory, B from shared memory
__device__ __forceinline__ void mma_bf16_ts(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accum)
{
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
                 "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accum), "r"(leader)
                 : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
                 "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
                 "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
                 "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
                 "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
                 : "memory");
}

// 16 bytes from global to shared memory, past L1
__device__ __forceinline__ void copy16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// one arrival of this thread (counted at the mbarrier's set-up) when its copies so far are complete
__device__ __forceinline__ void arrive_copied(uint32_t bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// 32 E2M1 codes times 2^(se - 127) -> 32 BF16 values, exactly, as pairs in the order (e0 e4) (e1 e5) (e2 e6) (e3 e7) of each
// eight (a code and the one four after it lie 16 bits apart, so one shift puts both at their places in a BF16 pair).  A
// code's exponent and mantissa bits at the low end of the BF16 exponent are its value times 2^-126; one multiply by
// 2^(se - 1) gives the value.  Scales past 2 (se > 128, whose factor has no BF16 form) take a second multiply, 255 (NaN)
// among them.
__device__ __forceinline__ void dequant32_e2m1(const uint4 &v, uint32_t se, uint32_t *o)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t f = (min(se, 128u) + 126u) << 7;
    f |= f << 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t h = w[i] >> 8;
        o[4 * i] = ((w[i] << 6) & 0x01C001C0u) | ((w[i] << 12) & 0x80008000u);
        o[4 * i + 1] = ((w[i] << 2) & 0x01C001C0u) | ((w[i] << 8) & 0x80008000u);
        o[4 * i + 2] = ((h << 6) & 0x01C001C0u) | ((w[i] << 4) & 0x80008000u);
        o[4 * i + 3] = ((h << 2) & 0x01C001C0u) | (w[i] & 0x80008000u);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
        o[i] = mul_bf16x2(o[i], f);
    if (se > 128u) {
        uint32_t g = se == 255u ? 0x7FC0u : (se - 1u) << 7;   // 2^(se - 128)
        g |= g << 16;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            o[i] = mul_bf16x2(o[i], g);
    }
}

// bytes of w by the selector's nibbles, those of 8 and more the sign of byte - 8, eight times
__device__ __forceinline__ uint32_t prmt(uint32_t w, uint32_t sel)
{
    uint32_t r;
    asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(w), "r"(sel));
    return r;
}

// two E4M3 codes times a scale -> a BF16 pair (exact for every code and scale; NaN codes stay NaN)
__device__ __forceinline__ uint32_t convert2_e4m3(uint32_t two, float scale)
{
    const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(two & 0xFFFFu), __NV_E4M3);
    const float2 f = __half22float2(__half2(hr));
    return pack_bf16x2(f.x * scale, f.y * scale);
}

__device__ __forceinline__ float scale_of(uint32_t se)   // 2^(se - 127); 255: NaN
{
    return se == 255u ? __int_as_float(0x7FC00000) : se == 0u ? __int_as_float(0x00400000) : __int_as_float((int)(se << 23));
}

// 64 E4M3 codes times 2^(se - 127) -> 64 BF16 values as pairs.  A code s.eeee.mmm placed as the BF16 pattern
// s.0000eeee.mmm0000 is its value times 2^-120; one multiply by 2^(se - 7) gives the value.  A byte and its sign eight
// times over, shifted by four (a multiplication: the logic pipe is the fuller one), has every bit in its place.  Chunks with
// the NaN code, or a scale past 2^7, take the hardware's conversion.
__device__ __forceinline__ void dequant64_e4m3(const uint4 (&v)[4], uint32_t se, uint32_t (&o)[32])
{
    uint32_t f = (min(se, 134u) + 120u) << 7, odd = 0u;
    f |= f << 16;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const uint32_t w = (i & 3) == 0 ? v[i >> 2].x : (i & 3) == 1 ? v[i >> 2].y : (i & 3) == 2 ? v[i >> 2].z : v[i >> 2].w;
        o[2 * i] = mul_bf16x2((prmt(w, 0x9180) * 16u) & 0x87F087F0u, f);
        o[2 * i + 1] = mul_bf16x2((prmt(w, 0xB3A2) * 16u) & 0x87F087F0u, f);
        odd |= (w & 0x7F7F7F7Fu) + 0x01010101u;   // (bit 7 of a byte: its magnitude was 0x7F)
    }
    if (se > 134u || (odd & 0x80808080u) != 0u) {
        const float sc = scale_of(se);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const uint32_t w = (i & 6) == 0 ? v[i >> 3].x : (i & 6) == 2 ? v[i >> 3].y : (i & 6) == 4 ? v[i >> 3].z : v[i >> 3].w;
            o[i] = convert2_e4m3(w >> (16 * (i & 1)), sc);
        }
    }
}

__device__ __forceinline__ int blocks_of(int len) { return (len + kBK - 1) / kBK; }

// The work of this CTA: [w, w1) of all tokens' blocks, in the order of the tokens, each token with `extra` blocks' worth of time
// before its first (its queries take the place of the last token's).  Every role walks the same blocks.
struct Walk {
    int w, w1, extra;
    int t, start;     // the next token, and where its work begins
};

struct Segment {
    int t, len;       // token, and its keys
    int kb, nb;       // blocks kb .. kb + nb - 1 of it
};

__device__ __forceinline__ bool next_segment(Walk &k, const KeyWeightsParams &p, Segment &s)
{
    while (k.start < k.w1) {    // (tokens without keys have no work)
        s.len = __ldcg(p.lens + k.t);
        s.t = k.t++;
        const int n = blocks_of(s.len), at = k.start + k.extra;
        s.kb = max(0, k.w - at);
        s.nb = min(n, k.w1 - at) - s.kb;
        k.start += n > 0 ? n + k.extra : 0;
        if (s.nb > 0)
            return true;
    }
    return false;
}

template <int kH, bool kFour>
__global__ void __launch_bounds__(kThreads, 1) key_weights_kernel(const KeyWeightsParams p)
{
    using S = Shape<kH, kFour>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];   // (the swizzled tiles of Q start on 1024-byte boundaries)
    constexpr int kDepth = S::kDepth;
    constexpr int kQChunkBytes = kH * 128;
    // instruction descriptor (kind::f16): D f32, A/B bf16, both K-major
    constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(kH >> 3) << 17) | ((uint32_t)(kBK >> 4) << 24);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sQ = smem_u32(smem_raw), sRaw = sQ + kChunks * kQChunkBytes;
    uint8_t *small = smem_raw + kChunks * kQChunkBytes + 4 * kDepth * S::kUnitBytes;
    float *slse = reinterpret_cast<float *>(small + kOffLse);
    const uint32_t bar_raw_full = smem_u32(small + kOffBars);  // [quadrant][unit] its entries are there
    const uint32_t bar_raw_empty = bar_raw_full + 32 * kMaxDepth;  // [quadrant][unit] dequantised (its nine chunks)
    const uint32_t bar_full = bar_raw_empty + 32 * kMaxDepth;  // [slot] the chunk is in tensor memory (a set's four warps)
    const uint32_t bar_empty = bar_full + 8 * kSlots;          // [slot] read by its products
    const uint32_t bar_dfull = bar_empty + 8 * kSlots;         // [2] the block's products are complete
    const uint32_t bar_dempty = bar_dfull + 16;                // [2] read by the epilogue
    const uint32_t bar_q = bar_dfull + 32;                     // [group] of the segment's Q is there
    const uint32_t bar_qfree = bar_q + 8 * kQGroups;           // [group] the segment's last products with it are done
    const uint32_t bar_qraw = bar_qfree + 8 * kQGroups;        // [group] copied (a later segment's)
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(small + kOffTmem);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(small + kOffAbort);
    int *first = reinterpret_cast<int *>(small + kOffStart);
    int2 *scan = reinterpret_cast<int2 *>(small + kOffLse);

    if (tid == 0) {
        for (int i = 0; i < 4 * kMaxDepth; ++i) {
            mbar_init(bar_raw_full + 8 * i, 32);
            mbar_init(bar_raw_empty + 8 * i, kSets);
        }
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(bar_full + 8 * i, 4);
            mbar_init(bar_empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar_dfull + 8 * i, 1);
            mbar_init(bar_dempty + 8 * i, kEpilogueWarps);
        }
        for (int i = 0; i < kQGroups; ++i) {
            mbar_init(bar_q + 8 * i, kKeyWarps);
            mbar_init(bar_qfree + 8 * i, 1);
            mbar_init(bar_qraw + 8 * i, 32);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        *abort_flag = 0;
    }
    // (only the list kernel can still be running ahead of this one: it waited for what came before)
    if (warp == 0)
        tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    {   // the queries of the token that the CTA begins with if all lists are equally long, while the lists are made
        const int t = (int)((long long)p.num_tokens * blockIdx.x / gridDim.x);
        const uint8_t *q = reinterpret_cast<const uint8_t *>(p.q + (int64_t)t * p.q_token_stride);
        for (int i = tid; i < (kH * kDim * 2 + 127) / 128; i += kThreads)
            prefetch_l2(q + 128 * i);
    }
    griddep_wait();

    // ---- this CTA's blocks
    Walk walk;
    {
        const int per = (p.num_tokens + kThreads - 1) / kThreads;
        const int t0 = min(p.num_tokens, tid * per), t1 = min(p.num_tokens, t0 + per);
        int mine = 0, mine_tokens = 0, n0 = 0;   // blocks, tokens with keys, blocks of the first
        for (int t = t0; t < t1; ++t) {
            const int n = blocks_of(__ldcg(p.lens + t));
            n0 = t == t0 ? n : n0;
            mine += n;
            mine_tokens += n > 0;
        }
        int incl = mine, incl_tokens = mine_tokens;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, d), z = __shfl_up_sync(0xffffffffu, incl_tokens, d);
            if (lane >= d) {
                incl += y;
                incl_tokens += z;
            }
        }
        if (lane == 31)
            scan[warp] = make_int2(incl, incl_tokens);
        __syncthreads();
        const int2 x = scan[min(lane, kThreads / 32 - 1)];
        const bool sum = lane < kThreads / 32, below = lane < warp;
        const int W = __reduce_add_sync(0xffffffffu, sum ? x.x : 0), tokens = __reduce_add_sync(0xffffffffu, sum ? x.y : 0);
        int at = incl - mine + __reduce_add_sync(0xffffffffu, below ? x.x : 0);
        const int at_tokens = incl_tokens - mine_tokens + __reduce_add_sync(0xffffffffu, below ? x.y : 0);
        walk.extra = W >= kLongRun * (int)gridDim.x ? kSwitch : 0;
        const unsigned all = W + tokens * walk.extra, each = all / gridDim.x, more = all % gridDim.x;
        walk.w = (int)(each * blockIdx.x + min(blockIdx.x, more));
        walk.w1 = walk.w + (int)(each + (blockIdx.x < more ? 1u : 0u));
        at += at_tokens * walk.extra;
        mine += mine_tokens * walk.extra;
        if (walk.w < walk.w1 && mine > 0 && at <= walk.w && walk.w < at + mine) {
            int t = t0;
            for (int n = n0; at + (n > 0 ? n += walk.extra : 0) <= walk.w; n = blocks_of(__ldcg(p.lens + t))) {
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
        walk.start = walk.w < walk.w1 ? first[1] : walk.w1;
    }
    const uint32_t tmem = *tmem_slot;
    griddep_launch();   // (the adding kernel waits for this grid itself)
    Segment seg;
    uint32_t g = 0;     // blocks since the kernel began

    if (warp == 0) {
        // ---- the products: K-major operands advance 32 B, or eight columns, per 16 dims
        const uint32_t leader = elect_one();
        const uint64_t db = sdesc(sQ, 16, 1024);
        uint32_t at = 0;   // chunks since the kernel began
        for (uint32_t n = 0; next_segment(walk, p, seg); ++n) {
            for (int b = 0; b < seg.nb; ++b, ++g) {
                const uint32_t x = g & 1u;
                if (g >= 2) {
                    mbar_wait(bar_dempty + 8 * x, ((g >> 1) - 1) & 1u, abort_flag, p.status);
                    after_sync();
                }
#pragma unroll 3
                for (int c = 0; c < kChunks; ++c, ++at) {
                    const uint32_t slot = at % kSlots;
                    if (b == 0 && c % 3 == 0)
                        mbar_wait(bar_q + 8 * (c / 3), n & 1u, abort_flag, p.status);
                    mbar_wait(bar_full + 8 * slot, (at / kSlots) & 1u, abort_flag, p.status);
                    after_sync();
                    const uint64_t bq = db + (uint64_t)(((c + kChunks - 1) % kChunks * kQChunkBytes) >> 4);   // (the rope dims first)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_bf16_ts(leader, tmem + kH * x, tmem + kColKeys + 32 * slot + 8 * k, bq + (uint64_t)(2 * k), kIdesc,
                                    (c != 0 || k != 0) ? 1u : 0u);
                    commit(leader, bar_empty + 8 * slot);
                    if (b == seg.nb - 1 && c % 3 == 2)
                        commit(leader, bar_qfree + 8 * (c / 3));
                }
                commit(leader, bar_dfull + 8 * x);
            }
        }
    } else if (warp <= kEpilogueWarps) {
        // ---- sums over the heads: lane l of quadrant q has key 32 q + l of the block
        const int quad = warp & 3, row = 32 * quad + lane;
        const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
        const float c2 = p.scale * 1.4426950408889634f;
        while (next_segment(walk, p, seg)) {
            const int t = seg.t;
            const int r = p.req_idx != nullptr ? __ldcg(p.req_idx + t) : t;
            const bool first_of = __ldcg(p.later + t) == 0;
            named_bar(1, 32 * kEpilogueWarps);   // (slse has been read)
            bool without = false;
            if (row < kH) {
                const float l = __ldcg(p.lse + (int64_t)t * kH + row);
                without = l == -INFINITY;
                const float m = l * -1.4426950408889634f;
                slse[row] = without ? INFINITY : m == INFINITY ? 0x1.fffffep127f : m;
            }
            const bool some_without = named_bar_or(1, 32 * kEpilogueWarps, without);   // (heads that give nothing, whatever their logits)
            // the place of a block's key (-1: none), read a block ahead
            const int64_t list = (int64_t)t * p.list_w;
            auto load_place = [&](int b) {
                const int i = (seg.kb + b) * kBK + row;
                return b < seg.nb && i < seg.len ? __ldcg(p.positions + list + i) : -1;
            };
            float *row_out = p.weights + (int64_t)max(r, 0) * p.weights_stride;
            int place_next = load_place(0);
            for (int b = 0; b < seg.nb; ++b, ++g) {
                const uint32_t x = g & 1u;
                const int place = place_next;
                const float had = first_of && place >= 0 ? __ldcg(row_out + place) : 0.f;
                place_next = load_place(b + 1);
                mbar_wait(bar_dfull + 8 * x, (g >> 1) & 1u, abort_flag, p.status);
                after_sync();
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
                if (some_without) {
#pragma unroll 1
                    for (int h = 0; h < kH; h += 16) {
                        uint32_t s[16];
                        tmem_ld16(lane_base + kH * x + h, s);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const float l = slse[h + j];
                            sum[j & 3] += l == INFINITY ? 0.f : exp2_approx(fmaf(__uint_as_float(s[j]), c2, l));
                        }
                    }
                } else
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
                const float weight = (sum[0] + sum[1]) + (sum[2] + sum[3]);
                if (!first_of && (seg.kb + b) * kBK + row < seg.len)
                    __stcg(p.got + list + (seg.kb + b) * kBK + row, weight);
                else if (place >= 0)
                    __stcg(row_out + place, had + weight);
            }
        }
    } else if (warp < kKeyWarp0) {
        // ---- the entries of two quadrants, four lanes to a row (rows without a key keep what was there: nobody reads their
        // sums): a lane has the rows lane / 4, + 8, + 16 and + 24 of a quadrant, whose addresses are all that it computes.  Every
        // unit of a ring is filled by one warp, so it is never two phases behind its barrier
        constexpr int kPieces = S::kEntry / 16;
        const int quad0 = 2 * (warp - kCopyWarp0);
        const uint8_t *kv = p.kv + 16 * (lane & 3);
        const uint32_t dst0 = sRaw + (lane >> 2) * S::kEntry + 16 * (lane & 3);
        uint32_t unit = 0, round = 0;   // the next unit of the two rings, and how often they have been filled
        while (next_segment(walk, p, seg)) {
            const int32_t *list = p.slots + (int64_t)seg.t * p.list_w;
            int next[2][4];
            auto load_slots = [&](int b) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int i = ((seg.kb + b) * 4 + quad0 + j) * 32 + 8 * k + (lane >> 2);
                        next[j][k] = b < seg.nb && i < seg.len ? __ldcg(list + i) : -1;
                    }
            };
            load_slots(0);
            for (int b = 0; b < seg.nb; ++b) {
                int slot[2][4];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    slot[i >> 2][i & 3] = next[i >> 2][i & 3];
                load_slots(b + 1);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint32_t at_unit = (quad0 + j) * kDepth + unit;
                        if (round > 0)
                            mbar_wait(bar_raw_empty + 8 * at_unit, (round - 1) & 1u, abort_flag, p.status);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int from = slot[j][2 * half + k];
                            if (from < 0)
                                continue;
                            const uint8_t *src = kv + (int64_t)from * S::kEntry;
                            const uint32_t dst = dst0 + at_unit * S::kUnitBytes + 8 * k * S::kEntry;
#pragma unroll
                            for (int i = 0; i < kPieces / 4; ++i)
                                copy16(dst + 64 * i, src + 64 * i);
                            if ((lane & 3) < kPieces % 4)
                                copy16(dst + kPieces / 4 * 64, src + kPieces / 4 * 64);
                        }
                        arrive_copied(bar_raw_full + 8 * at_unit);
                    }
                    if (++unit == kDepth) {
                        unit = 0;
                        ++round;
                    }
                }
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp < kQWarp) {
        // ---- the keys: lane l of quadrant q has key 32 q + l of the block.  A set has two latent chunks of it, the first set the
        // rope dims as well, which need no conversion.  All are taken out of the ring at once, so that it fills again meanwhile
        const int kw = warp - kKeyWarp0, set = kw >> 2, quad = warp & 3;
        const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16) + kColKeys;
        const int c0 = (set + 3) & 3;   // its latent chunks: c0 and c0 + 4
        constexpr int kRaw = kFour ? 2 : 4;
        uint32_t blk = 0;        // blocks since the kernel began
        // a chunk into the next slot (blk * kChunks + m is its number)
        auto put = [&](const uint32_t (&o)[32], int m) {
            const uint32_t at = blk * kChunks + m, slot = at % kSlots;
            if (at >= kSlots) {
                mbar_wait(bar_empty + 8 * slot, ((at / kSlots) & 1u) ^ 1u, abort_flag, p.status);
                after_sync();
            }
            tmem_st32(lane_base + 32 * slot, o);
            tmem_st_wait();
            before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar_full + 8 * slot);
        };
        // 16 bytes of Q in the order of the latent dims that dequant32_e2m1 gives
        auto order_q = [&](uint32_t a) {
            const uint4 x = lds16(a);
            st_shared_v4(a, __byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632), __byte_perm(x.y, x.w, 0x5410),
                         __byte_perm(x.y, x.w, 0x7632));
        };
        for (uint32_t n = 0; next_segment(walk, p, seg); ++n) {
            const uint32_t first_block = blk;
            if (n == 0) {   // the first Q by all of these warps: their entries are not there yet
                const uint4 *q = reinterpret_cast<const uint4 *>(p.q + (int64_t)seg.t * p.q_token_stride);
                auto place = [&](int i) {   // of the i-th 16 bytes of Q
                    const int h = i / (kDim / 8), c = i % (kDim / 8);
                    return sQ + (c >> 3) * kQChunkBytes + sw128(h, c & 7);
                };
                for (int i = 32 * kw + lane; i < kH * (kDim / 8); i += 32 * kKeyWarps)
                    copy16(place(i), q + i);
                asm volatile("cp.async.wait_all;" ::: "memory");
                if (kFour)   // (each thread its own pieces)
                    for (int i = 32 * kw + lane; i < kH * (kDim / 8); i += 32 * kKeyWarps)
                        if (i % (kDim / 8) < kLatent / 8)
                            order_q(place(i));
                fence_async_smem();
                __syncwarp();
                if (lane < kQGroups)
                    mbar_arrive(bar_q + 8 * lane);
            }
            g += (uint32_t)seg.nb;
            for (; blk < g; ++blk) {
                // both units of the quadrant's half blocks, and this lane's entry in its own
                const uint32_t u0 = 2 * blk, u1 = 2 * blk + 1;
                const uint32_t unit0 = quad * kDepth + u0 % kDepth, unit1 = quad * kDepth + u1 % kDepth;
                mbar_wait(bar_raw_full + 8 * unit0, (u0 / kDepth) & 1u, abort_flag, p.status);
                mbar_wait(bar_raw_full + 8 * unit1, (u1 / kDepth) & 1u, abort_flag, p.status);
                const uint32_t e = sRaw + (lane < 16 ? unit0 : unit1) * S::kUnitBytes + (lane & 15) * S::kEntry;
                uint4 v[2][kRaw];
                uint32_t se[2][2], o[32];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int c = c0 + 4 * j;
#pragma unroll
                    for (int i = 0; i < kRaw; ++i)
                        v[j][i] = lds16(e + 16 * (kRaw * c + i));
                    se[j][0] = lds8(e + (kFour ? kScale4Offset + 2 * c : kScaleOffset + (c >> 1)));
                    se[j][1] = kFour ? lds8(e + kScale4Offset + 2 * c + 1) : 0u;
                }
                if (set == 0)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint4 x = lds16(e + (kFour ? kRope4Offset : kRopeOffset) + 16 * i);
                        o[4 * i] = x.x;
                        o[4 * i + 1] = x.y;
                        o[4 * i + 2] = x.z;
                        o[4 * i + 3] = x.w;
                    }
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar_raw_empty + 8 * unit0);
                    mbar_arrive(bar_raw_empty + 8 * unit1);
                }
                if (set == 0)
                    put(o, 0);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if constexpr (kFour) {
                        dequant32_e2m1(v[j][0], se[j][0], o);
                        dequant32_e2m1(v[j][1], se[j][1], o + 16);
                    } else {
                        dequant64_e4m3(v[j], se[j][0], o);
                    }
                    put(o, c0 + 1 + 4 * j);
                    // a later segment's Q, after the chunks that go into tensor memory without its products
                    if (n > 0 && j == 0 && blk == first_block)
                        for (int grp = 0; grp < kQGroups; ++grp) {
                            mbar_wait(bar_qraw + 8 * grp, (n - 1) & 1u, abort_flag, p.status);
                            if (kFour)
                                for (int i = (grp == 0 ? 8 * kH : 0) + 32 * kw + lane; i < 3 * 8 * kH; i += 32 * kKeyWarps)
                                    order_q(sQ + (3 * grp - 1) * kQChunkBytes + 16 * i);
                            fence_async_smem();
                            __syncwarp();
                            if (lane == 0)
                                mbar_arrive(bar_q + 8 * grp);
                        }
                }
            }
        }
    } else {
        // ---- the Q of later segments, a group of chunks as soon as the products of the segment before are done with it
        for (uint32_t n = 0; next_segment(walk, p, seg); ++n) {
            const uint16_t *q = p.q + (int64_t)seg.t * p.q_token_stride + (lane >> 3) * kDim + 8 * (lane & 7);
#pragma unroll 1
            for (int grp = 0; grp < kQGroups && n > 0; ++grp) {
                mbar_wait(bar_qfree + 8 * grp, (n - 1) & 1u, abort_flag, p.status);
#pragma unroll 1
                for (int m = 3 * grp; m < 3 * grp + 3; ++m) {
                    const int c = m == 0 ? kChunks - 1 : m - 1;
                    const uint32_t dst = sQ + c * kQChunkBytes;
#pragma unroll 8
                    for (int h = 0; h < kH; h += 4)
                        copy16(dst + sw128(h + (lane >> 3), lane & 7), q + h * kDim + 64 * c);
                }
                arrive_copied(bar_qraw + 8 * grp);
            }
            if (walk.start < walk.w1) {   // the next token's
                const uint8_t *next = reinterpret_cast<const uint8_t *>(p.q + (int64_t)(seg.t + 1) * p.q_token_stride);
                for (int i = lane; i < (kH * kDim * 2 + 127) / 128; i += 32)
                    prefetch_l2(next + 128 * i);
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    }
    before_sync();
    __syncthreads();
    after_sync();
    if (warp == 0)
        tmem_free(tmem, kTmemCols);
}

// The tokens after a row's first one, in order.  One of them: the slices share its list.  Several: one after the other, positions
// dealt out to the slices in runs of 256.  What the list kernel wrote was complete before the one with the products let this one
// begin, so a thread has the positions of its first kFront entries before it waits for that one.
__global__ void __launch_bounds__(kAddThreads) add_weights_kernel(const KeyWeightsParams p)
{
    __shared__ int tokens[kAddThreads], wcount[kAddThreads / 32];
    const int slice = blockIdx.x % kAddSlices, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    bool waited = false;
    auto wait = [&]() {
        if (!waited) {
            griddep_wait();
            griddep_launch();
        }
        waited = true;
    };
    for (int64_t r = blockIdx.x / kAddSlices; r < p.num_reqs; r += gridDim.x / kAddSlices) {
        float *row = p.weights + r * p.weights_stride;
        for (int t0 = 0; t0 < p.num_tokens; t0 += kAddThreads) {
            const int t = min(t0 + tid, p.num_tokens - 1);
            const int of = p.req_idx[t], after = __ldcg(p.later + t);
            const bool mine = t == t0 + tid && of == r && after != 0;
            const unsigned m = __ballot_sync(0xffffffffu, mine);
            if (lane == 0)
                wcount[warp] = __popc(m);
            __syncthreads();
            int before = 0, all = 0;
            for (int w = 0; w < kAddThreads / 32; ++w) {
                before += w < warp ? wcount[w] : 0;
                all += wcount[w];
            }
            if (mine)
                tokens[before + __popc(m & ((1u << lane) - 1u))] = t;
            __syncthreads();
            const bool deal = all > 1 || p.num_tokens > kAddThreads;   // (else it is the row's only one)
            const int begin = deal ? tid : slice * kAddThreads + tid, step = deal ? kAddThreads : kAddSlices * kAddThreads;
            for (int k = 0; k < all; ++k) {
                const int token = tokens[k], len = __ldcg(p.lens + token);
                const int64_t at = (int64_t)token * p.list_w;
                int64_t i0 = begin;
                do {
                    int pos[kFront];
                    float got[kFront], had[kFront];
#pragma unroll
                    for (int u = 0; u < kFront; ++u) {
                        const int64_t i = i0 + u * step;
                        pos[u] = __ldcg(p.positions + at + min(i, (int64_t)p.list_w - 1));   // (beside the length)
                        if (i >= len || (deal && (pos[u] >> 8) % kAddSlices != slice))
                            pos[u] = -1;
                        if (pos[u] >= 0)
                            prefetch_l2(row + pos[u]);
                    }
                    wait();
#pragma unroll
                    for (int u = 0; u < kFront; ++u) {
                        got[u] = pos[u] >= 0 ? __ldcg(p.got + at + i0 + u * step) : 0.f;
                        had[u] = pos[u] >= 0 ? __ldcg(row + pos[u]) : 0.f;
                    }
#pragma unroll
                    for (int u = 0; u < kFront; ++u)
                        if (pos[u] >= 0)
                            __stcg(row + pos[u], had[u] + got[u]);
                    i0 += kFront * step;
                } while (i0 < len);
                __syncthreads();   // the next token's sums come on top
            }
            __syncthreads();
        }
    }
    wait();
}

template <int kH, bool kFour>
cudaError_t launch(const KeyWeightsParams &p, int sms, cudaStream_t stream)
{
    const auto kernel = key_weights_kernel<kH, kFour>;
    constexpr int kSlot = kAttrKeyWeights + (kH == 16 ? 0 : kH == 32 ? 1 : kH == 64 ? 2 : 3) + (kFour ? 4 : 0);
    const cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kernel), Shape<kH, kFour>::kSmem, (AttrSlot)kSlot);
    if (e != cudaSuccess)
        return e;
    const long long blocks = (long long)p.num_tokens * ((p.list_w + kBK - 1) / kBK);   // at most
    return launch_dependent(kernel, dim3((unsigned)std::min<long long>(sms, blocks)), kThreads, Shape<kH, kFour>::kSmem, stream, p);
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
    return launch_dependent(add_weights_kernel, dim3(kAddSlices * (unsigned)std::min(p.num_reqs, kAddRows)), kAddThreads, 0, stream, p);
}

}  // namespace dsv4
