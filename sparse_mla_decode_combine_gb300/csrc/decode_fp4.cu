// decode_fp4.cu -- sparse-MLA decode over the 4-bit cache on the tensor cores (tcgen05 / TMEM).
//
// Operation (per token t, head h, over the token's combined list of positions):
//   s_p = scale * q_h . k_p (576 dims),  lse_h = ln(sum_p e^{s_p} + e^{sink_h}),  out_h = sum_p e^{s_p - lse_h} v_p
// The lists of cache slots come from the list kernel (lists_fp4.cu) ahead of this one in the stream.
//
// Contraction.  All heads share one key set, so a (token, 64 heads) unit is a pair of dense products, run
// transposed (keys and value dims on the M side of the tensor tile):
//   S^T[64 keys x 64 heads]   = K_tile[64 x 576] . Q^T          (A = K tile, K-major)
//   O^T[128 dv x 64 heads]   += V^T[128 dv x 64 keys] . P^T     (A = the same bytes, MN-major), four tiles
// A K tile is a dequantised block in BF16 (exact: an E2M1 code times a power of two), nine 64-dim column
// chunks of 128-byte-swizzled rows: 74 KB, twice, beside the 74 KB of Q.
//
// Pipeline over two K tiles.  While the workers do the softmax of block b in one tile, S^T of block b + 1 runs
// from the other; while they write block b + 2 over block b (behind P.V of b, half the value dims at a time),
// P.V of b runs.  What the tensor cores read (a product of M 128 or 64 x N 64 x K 16 takes 6 or 4 KB of
// operands) and what the workers write share 128 B a cycle of shared memory: about 5 k cycles for 128 keys,
// which bounds a long list.  (One 128-key tile, whose steps form a chain, took 8.5 k.)
//   - a thread holds its eighth of a row's next entry in registers, loaded as those of the present block are
//     used up; whole entries are prefetched to L2 two blocks before that;
//   - the softmax keeps a reference maximum per head from the unit's first block and exchanges maxima between
//     warps again only when a logit exceeds it by 2^40: P and the sums are floating-point numbers, whose
//     relative precision does not depend on the reference, and 2^40 is far from fp32's and BF16's range.  The
//     usual block needs one barrier that ORs a predicate.  Row sums stay in registers.
//
// CTA = 26 warps for one (token, 64-head group, split): warp 0 issues S^T, warp 25 P.V, warps 1-8 do the softmax,
// warps 9-24 the dequant and the epilogue.  16 or 32 heads run as a 64-head group whose missing
// heads have zero queries (their columns are computed and dropped).  The splits of a unit form a cluster and
// merge through distributed shared memory.  Every mbarrier wait is bounded.
//
// Order of the dims inside a tile.  The eight 4-bit codes of a 32-bit word become the pairs (e_k, e_{k+4}):
// code k and code k + 4 lie 16 bits apart, so one shift puts both at their places in a BF16 pair (two masked
// shifts: magnitude and sign).  Inside each group of eight latent dims the tile therefore holds e0 e4 e1 e5 e2
// e6 e3 e7; Q is stored in the same order, and the epilogue writes each value dim to its own place.
#include <climits>
#include <cuda_bf16.h>
#include <math.h>

#include "fp4.h"
#include "tcgen05.cuh"

namespace dsv4 {
namespace {

using namespace tc;

constexpr int kSoftmaxWarps = 8;         // warps 1-8 (warp 0 issues S^T)
constexpr int kDequantWarp0 = 9;
constexpr int kDequantWarps = 16;        // warps 9-24: also Q's layout and the epilogue
constexpr int kPvWarp = 25;              // issues P.V
constexpr int kThreads = 832;
constexpr int kWorkers = 32 * kDequantWarps;
constexpr int kBK = 64;                  // keys per block = MMA M of the logits
constexpr int kDvTile = 128;             // value dims per tile = MMA M of P.V
constexpr int kNH = 64;                  // heads per CTA = MMA N
constexpr int kChunks = 9;               // 576 dims / 64
constexpr int kQBytes = kChunks * kNH * 128;     // 73728
constexpr int kKBytes = kChunks * kBK * 128;     // 73728: one of two K tiles
constexpr int kChunkBytes = kBK * 128;           // 8192 (one 64-dim column chunk of a K tile)
constexpr int kQChunkBytes = kNH * 128;          // 8192
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0;            // S^T: 64 columns for each of the two K tiles
constexpr uint32_t kColO = 128;          // O^T: 4 tiles x 64 columns
constexpr float kExceedLog2 = 40.f;
constexpr int kMaxSplits = 8;            // portable cluster size

// small shared region (after Q and the two K tiles)
constexpr int kOffRed = 0;               // float [4][64]: per-quadrant head maxima, or row sums at the end
constexpr int kOffMax = 1024;            // float [64]: reference maximum per head (log2 units; natural ones at the end)
constexpr int kOffFin = 1280;            // float [64]: the factor of a rescale; at the end the output's, or a split's row sum
constexpr int kOffValid = 1536;          // uint8 [2][64]: rows of a K tile that hold a key
constexpr int kOffBars = 1664;           // u64: bar_s[2], bar_p[2], bar_grp[2][2], bar_pv[2][4]
constexpr int kOffTmem = 1792;           // u32
constexpr int kOffAbort = 1796;          // int
constexpr int kSmallBytes = 1856;
constexpr int kSmemBytes = kQBytes + 2 * kKBytes + kSmallBytes + 1024;   // + alignment slack
constexpr int kQLoads = kNH * (kDim / 8) / kWorkers;                     // 9 16-byte Q pieces per worker
static_assert(kNH * (kDim / 8) % kWorkers == 0, "Q pieces per worker");
static_assert(2 * kKBytes >= (kNH + kMaxSplits) * kLatent * (int)sizeof(float), "the partials fit the K tiles");

// instruction descriptors (kind::f16): D f32, A/B bf16, N = 64
constexpr uint32_t kIdescBase = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(kNH >> 3) << 17);
constexpr uint32_t kIdescQK = kIdescBase | ((uint32_t)(kBK >> 4) << 24);                              // A, B K-major
constexpr uint32_t kIdescPV = kIdescBase | ((uint32_t)(kDvTile >> 4) << 24) | (1u << 15) | (1u << 16);   // A, B MN-major

// 16 bytes of an entry.  Entries start at odd multiples of 16 bytes as often as at even ones, so a row's 64-byte
// pieces share 32-byte sectors with their neighbours: L1 keeps them for the next piece (8 % of the kernel's time
// against loads that do not allocate there).
__device__ __forceinline__ uint4 ld16(const void *p) { return __ldg(reinterpret_cast<const uint4 *>(p)); }

// 32 E2M1 codes times 2^(se - 127) -> 16 BF16 pairs, exactly.
// A code's exponent and mantissa bits at the low end of the BF16 exponent are its value times 2^-126 (both
// formats put the binary point the same way, subnormals included); one multiply by 2^(se - 1) gives the value.
// Scales past 2 (se > 128, whose factor has no BF16 form) take a second multiply, 255 (NaN) among them.
__device__ __forceinline__ void dequant32(const uint4 &v, uint32_t se, uint32_t (&o)[16])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t f = (min(se, 128u) + 126u) << 7;
    f |= f << 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t u = w[i] >> 8;
        o[4 * i + 0] = ((w[i] << 6) & 0x01C001C0u) | ((w[i] << 12) & 0x80008000u);
        o[4 * i + 1] = ((w[i] << 2) & 0x01C001C0u) | ((w[i] << 8) & 0x80008000u);
        o[4 * i + 2] = ((u << 6) & 0x01C001C0u) | ((w[i] << 4) & 0x80008000u);
        o[4 * i + 3] = ((u << 2) & 0x01C001C0u) | (w[i] & 0x80008000u);
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

// Split merge inside a cluster of S CTAs (one per split of a token's keys).  The CTA of rank r owns heads
// [r*hp, (r+1)*hp), hp = ceil(64 / S).  Every split s has pushed, into each owner's shared memory, its reference
// maximum m_s (natural-log units, -inf for a split without keys) and row sum l_s for the owner's heads
// (stat[s][hl] = (m_s, l_s)) and its unnormalised fp32 O_s (recv[s][hl][512]).  The owner forms
//   m = max(max_s m_s, sink), Z = sum_s l_s e^{m_s - m} + e^{sink - m},
//   out = sum_s e^{m_s - m} O_s / Z  (BF16),  lse = m + ln Z.
__device__ __noinline__ void merge_splits(uint16_t *out, float *lse, const float *sink, int num_heads, int S, int t,
                                          int h0, int rank, const float *recv, const float *stat, float *wts)
{
    const int hp = (kNH + S - 1) / S;
    const int hb = rank * hp;
    const int nh = max(0, min(min(kNH, num_heads - h0), hb + hp) - hb);   // owned heads that exist
    const int tid = threadIdx.x;
    if (tid < nh) {
        float mk = -INFINITY;
        for (int s = 0; s < S; ++s)
            mk = fmaxf(mk, stat[2 * (s * hp + tid)]);
        const float sk = sink != nullptr ? sink[h0 + hb + tid] : -INFINITY;
        const float m = fmaxf(mk, sk);
        float z = sk == -INFINITY ? 0.f : expf(sk - m);
        for (int s = 0; s < S; ++s) {
            const float ms = stat[2 * (s * hp + tid)];
            const float w = ms == -INFINITY ? 0.f : expf(ms - m);
            wts[tid * 10 + s] = w;
            z += ms == -INFINITY ? 0.f : stat[2 * (s * hp + tid) + 1] * w;
        }
        const float f = mk == -INFINITY ? 0.f : 1.f / z;
        for (int s = 0; s < S; ++s)
            wts[tid * 10 + s] *= f;
        wts[tid * 10 + 8] = m == -INFINITY ? -INFINITY : m + logf(z);
    }
    __syncthreads();
    const int items = nh * (kLatent / 4);   // 16-byte pieces of the slice
    for (int i = tid; i < items; i += kThreads) {
        const int hl = i / (kLatent / 4);
        const int c = i % (kLatent / 4);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s = 0; s < S; ++s) {
            const float ws = wts[hl * 10 + s];
            if (ws != 0.f) {   // (a split without keys has sent nothing)
                const float4 v = *reinterpret_cast<const float4 *>(recv + ((size_t)(s * hp + hl)) * kLatent + 4 * c);
                acc.x = fmaf(ws, v.x, acc.x);
                acc.y = fmaf(ws, v.y, acc.y);
                acc.z = fmaf(ws, v.z, acc.z);
                acc.w = fmaf(ws, v.w, acc.w);
            }
        }
        const int64_t row = (int64_t)t * num_heads + h0 + hb + hl;
        *reinterpret_cast<uint2 *>(out + row * kLatent + 4 * c) = make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
        if (c == 0 && lse != nullptr)
            lse[row] = wts[hl * 10 + 8];
    }
}

// Sends the (m, l) pair of head h (0..63) of split `split` to the head's owner in the cluster.
__device__ __forceinline__ void push_stat(uint32_t stat_s, int S, int split, int h, float m, float l)
{
    const int hp = (kNH + S - 1) / S;
    const int r = h / hp;
    st_cluster_v2(map_to_rank(stat_s + (uint32_t)(2 * (split * hp + (h - r * hp))) * 4u, (uint32_t)r), m, l);
}

__global__ void __launch_bounds__(kThreads, 1) decode_fp4_kernel(const Decode4Params p)
{
    extern __shared__ uint8_t smem_raw[];
    const int tid = threadIdx.x;
    const int warp = tid >> 5;
    const int lane = tid & 31;
    const int split = blockIdx.x % p.splits;   // = rank in the cluster when splits > 1
    const int unit = blockIdx.x / p.splits;
    const int t = unit / p.groups;
    const int h0 = unit % p.groups * kNH;
    const int nhv = min(kNH, p.num_heads - h0);   // heads of the group that exist
    const bool is_worker = warp >= kDequantWarp0 && warp < kDequantWarp0 + kDequantWarps;
    const int ww = warp - kDequantWarp0;
    const int wid = tid - 32 * kDequantWarp0;     // worker index 0..511

    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;   // the swizzled tiles start on 1024-byte boundaries
    uint8_t *gbase = smem_raw + (base - raw);
    const uint32_t sQ = base;
    const uint32_t sK = base + kQBytes;           // two K tiles; P^T takes a tile's rope chunk once its S^T is done
    uint8_t *small = gbase + kQBytes + 2 * kKBytes;
    float *red = reinterpret_cast<float *>(small + kOffRed);
    float *smax = reinterpret_cast<float *>(small + kOffMax);
    float *fin = reinterpret_cast<float *>(small + kOffFin);
    uint8_t *valid = small + kOffValid;
    const uint32_t bar_s = smem_u32(small + kOffBars);   // [tile] S^T complete
    const uint32_t bar_p = bar_s + 16;                   // [tile] P^T written (softmax warps)
    const uint32_t bar_grp = bar_s + 32;                 // [tile][2] column chunks 0-3, then 4-8 written (dequant warps)
    const uint32_t bar_pv = bar_s + 64;                  // [tile][4] P.V of value tile m complete
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(small + kOffTmem);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(small + kOffAbort);

    // ---- set-up that does not read the lists
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar_s + 8 * i, 1);
            mbar_init(bar_p + 8 * i, kSoftmaxWarps);
        }
        for (int i = 0; i < 4; ++i)
            mbar_init(bar_grp + 8 * i, kDequantWarps);
        for (int i = 0; i < 8; ++i)
            mbar_init(bar_pv + 8 * i, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        *abort_flag = 0;
    }
    if (tid < kNH)
        smax[tid] = 0.f;
    if (warp == 0)
        tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    // Q into registers.  Only the lists come from the previous kernel, which began after everything before it in the
    // stream had ended: whatever else the call reads is there already.
    uint4 qv[kQLoads];
    if (is_worker) {
#pragma unroll
        for (int j = 0; j < kQLoads; ++j) {
            const int i = wid + kWorkers * j;
            const int h = i / (kDim / 8), c = i % (kDim / 8);
            qv[j] = make_uint4(0u, 0u, 0u, 0u);   // (zeros for heads that do not exist)
            if (h < nhv)
                qv[j] = __ldg(reinterpret_cast<const uint4 *>(p.q + (int64_t)t * p.q_token_stride + (int64_t)(h0 + h) * kDim + 8 * c));
        }
    }

    // Dequant: eight threads to a row, each with two 16-byte pieces of codes (32 dims each), one of rope and two scale
    // bytes.  Lanes 8 i .. 8 i + 7 of a warp take one eighth of eight rows whose numbers differ mod 8 (no bank conflicts
    // in the swizzled stores) and spread over the tile, so that a short block keeps every warp at work.
    const int eighth = 4 * (ww & 1) + (lane >> 3);
    const int rrow = 8 * (((ww >> 1) - (lane & 7)) & 7) + (lane & 7);
    const int32_t *list = p.slots + (int64_t)t * p.list_w;
    const int kbeg = split * p.chunk;
    uint4 pre[2], prope;   // the entry of the block ahead
    uint32_t psc[2];
    bool pre_ok = false;
    auto load_piece = [&](const uint8_t *e, int m) {
        pre[m] = ld16(e + 128 * m + 16 * eighth);
        psc[m] = __ldg(e + kScale4Offset + 8 * m + eighth);
    };
    auto load_rope = [&](const uint8_t *e) { prope = ld16(e + kRope4Offset + 16 * eighth); };
    auto entry = [&](int slot) { return p.kv + (int64_t)(slot >= 0 ? slot : 0) * kEntry4Bytes; };

    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int kend = min(p.lens[t], kbeg + p.chunk);
    const int nkeys = max(0, kend - kbeg);
    const int nblocks = (nkeys + kBK - 1) / kBK;
    // the cache slot of this thread's row in block b; -1 past the list's end
    auto slot_of = [&](int b) {
        const int i = kbeg + b * kBK + rrow;
        return i < kend ? __ldg(list + i) : -1;
    };
    int slot1 = -1, slot2 = -1;   // of the blocks ahead
    if (is_worker) {
        const int slot0 = slot_of(0);
        slot1 = slot_of(1);
        slot2 = slot_of(2);
        pre_ok = slot0 >= 0;
        if (pre_ok) {
            load_piece(entry(slot0), 0);
            load_piece(entry(slot0), 1);
            load_rope(entry(slot0));
        }
        // Q -> swizzled K-major B operand, in the tile's order of dims
#pragma unroll
        for (int j = 0; j < kQLoads; ++j) {
            const int i = wid + kWorkers * j;
            const int h = i / (kDim / 8), c = i % (kDim / 8);
            const uint32_t a = sQ + (c >> 3) * kQChunkBytes + sw128(h, c & 7);
            if (c < kLatent / 8)
                st_shared_v4(a, __byte_perm(qv[j].x, qv[j].z, 0x5410), __byte_perm(qv[j].x, qv[j].z, 0x7632),
                             __byte_perm(qv[j].y, qv[j].w, 0x5410), __byte_perm(qv[j].y, qv[j].w, 0x7632));
            else
                st_shared_v4(a, qv[j].x, qv[j].y, qv[j].z, qv[j].w);
        }
    }
    fence_async_smem();
    before_sync();
    __syncthreads();   // Q, barriers, TMEM address
    after_sync();
    const uint32_t tmem = *tmem_slot;

    if (nblocks == 0) {   // no key in this split
        if (warp == 0)
            tmem_free(tmem, kTmemCols);
        if (p.splits == 1) {   // zero output, the lse from the sink alone
            if (tid < nhv && p.lse != nullptr)
                p.lse[(int64_t)t * p.num_heads + h0 + tid] = p.sink != nullptr ? p.sink[h0 + tid] : -INFINITY;
            for (int i = tid; i < nhv * kLatent / 8; i += kThreads)
                *reinterpret_cast<uint4 *>(p.out + ((int64_t)t * p.num_heads + h0) * kLatent + 8 * i) = make_uint4(0, 0, 0, 0);
            return;
        }
        cluster_sync();   // every split is past its products: partials may land
        if (tid < kNH)
            push_stat(smem_u32(gbase), p.splits, split, tid, -INFINITY, 0.f);
        cluster_sync();   // every partial has landed
        merge_splits(p.out, p.lse, p.sink, p.num_heads, p.splits, t, h0, split,
                     reinterpret_cast<const float *>(gbase + kQBytes), reinterpret_cast<const float *>(gbase),
                     reinterpret_cast<float *>(gbase + 2048));
        return;
    }

    const int quad = warp & 3;                            // TMEM lane quadrant of this warp
    const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
    const int vrow = quad * 32 + lane;                    // this lane's row of a value tile,
    const int dv0 = (vrow & ~7) | ((vrow >> 1) & 3) | ((vrow & 1) << 2);   // and its value dim (the tile's order of dims)

    if (warp == 0) {
        // descriptors: K-major operands advance 32 B per 16 dims and one column chunk per 64
        const uint32_t leader = elect_one();
        const uint64_t qk_a = sdesc(sK, 16, 1024);
        const uint64_t qk_b = sdesc(sQ, 16, 1024);
        for (int b = 0; b < nblocks; ++b) {
            const int x = b & 1;
            const uint32_t ph = (uint32_t)(b >> 1) & 1u;
            const uint64_t ax = qk_a + (uint64_t)((x * kKBytes) >> 4);
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                if (c == 0 || c == 4) {
                    mbar_wait(bar_grp + 16 * x + 2 * c, ph, abort_flag, p.status);
                    after_sync();
                }
                const uint64_t a = ax + (uint64_t)((c * kChunkBytes) >> 4);
                const uint64_t bq = qk_b + (uint64_t)((c * kQChunkBytes) >> 4);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_bf16(leader, tmem + kColS + 64 * x, a + (uint64_t)(2 * k), bq + (uint64_t)(2 * k), kIdescQK,
                             (c != 0 || k != 0) ? 1u : 0u);
            }
            commit(leader, bar_s + 8 * x);
        }
    } else if (warp == kPvWarp) {
        // MN-major operands advance 2 KB per 16 keys
        const uint32_t leader = elect_one();
        const uint64_t pv_a = sdesc(sK, kChunkBytes, 1024);
        const uint64_t pv_b = sdesc(sK + 8 * kChunkBytes, 1024, 1024);
        for (int b = 0; b < nblocks; ++b) {
            const int x = b & 1;
            mbar_wait(bar_p + 8 * x, (uint32_t)(b >> 1) & 1u, abort_flag, p.status);
            after_sync();
            const uint64_t off = (uint64_t)((x * kKBytes) >> 4);
            const int left = nkeys - b * kBK;   // 16-key steps without a key are left out
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const uint64_t a = pv_a + off + (uint64_t)((2 * m * kChunkBytes) >> 4);
#pragma unroll
                for (int kk = 0; kk < kBK / 16; ++kk)
                    if (16 * kk < left)
                        mma_bf16(leader, tmem + kColO + 64 * m, a + (uint64_t)(kk * 128), pv_b + off + (uint64_t)(kk * 128),
                                 kIdescPV, (b > 0 || kk > 0) ? 1u : 0u);
                commit(leader, bar_pv + 32 * x + 8 * m);   // releases K chunks 2m, 2m+1 (m = 3: also P^T)
            }
        }
    } else if (is_worker) {
        const uint32_t rb = (uint32_t)(rrow >> 3) * 1024u + (uint32_t)(rrow & 7) * 128u;
        const uint32_t x7 = (uint32_t)(rrow & 7);
        for (int b = 0; b < nblocks; ++b) {   // block b into its K tile (zeros for rows without a key)
            const int x = b & 1;
            const uint32_t ph = (uint32_t)((b >> 1) - 1) & 1u;
            const uint32_t tile = sK + (uint32_t)x * kKBytes + rb;
            const bool ok_next = slot1 >= 0;
            const uint8_t *en = entry(slot1);   // the next block's entry goes into the registers as they are used up
#pragma unroll
            for (int m = 0; m < 2; ++m) {   // dims 256 m + 32 eighth ..
                uint32_t o[16];
                if (pre_ok) {
                    dequant32(pre[m], psc[m], o);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        o[i] = 0u;
                }
                if (ok_next)
                    load_piece(en, m);
                if (b >= 2)
                    mbar_wait(bar_pv + 32 * x + 16 * m + 8, ph, abort_flag, p.status);   // P.V of block b - 2 is done with them
                if (m == 0 && eighth == 0)
                    valid[x * kBK + rrow] = pre_ok;
                const uint32_t cb = tile + (uint32_t)(4 * m + (eighth >> 1)) * kChunkBytes;
                const uint32_t u = 4u * (uint32_t)(eighth & 1);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    st_shared_v4(cb + (((u + i) ^ x7) << 4), o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                if (m == 1) {   // the rope chunk, whose place P^T had
                    if (!pre_ok)
                        prope = make_uint4(0u, 0u, 0u, 0u);
                    st_shared_v4(tile + 8u * kChunkBytes + (((uint32_t)eighth ^ x7) << 4), prope.x, prope.y, prope.z, prope.w);
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar_grp + 16 * x + 8 * m);
            }
            if (ok_next)
                load_rope(en);
            pre_ok = ok_next;
            slot1 = slot2;
            slot2 = slot_of(b + 3);
        }
    } else {
        const float c2 = p.scale * 1.4426950408889634f;   // logits in log2 units per raw dot product
        const int hw = 32 * ((warp - 1) >> 2);            // first of this warp's 32 heads; its 16 keys are the quadrant's
        const int slice_bar = 2 + ((warp - 1) >> 2);      // the four warps of these heads
        // this lane's keys are srow and srow + 8; its heads, j = 0..7:
        const int srow = 16 * quad + (lane >> 2);
        const int sh = hw + 2 * (lane & 3);
        auto head = [&](int j) { return sh + 16 * (j >> 2) + 8 * ((j >> 1) & 1) + (j & 1); };
        float l[8];                                       // row sums of those heads over this lane's keys
#pragma unroll
        for (int j = 0; j < 8; ++j)
            l[j] = 0.f;
        bool fresh = true;                                // no key has been seen: the references are not set

        for (int b = 0; b < nblocks; ++b) {
            const int x = b & 1;
            const uint32_t ph = (uint32_t)(b >> 1) & 1u;
            mbar_wait(bar_grp + 16 * x, ph, abort_flag, p.status);   // (complete by then: the rows' flags are visible)
            const bool kv[2] = {valid[x * kBK + srow] != 0, valid[x * kBK + srow + 8] != 0};   // (not past the list's end)
            float ref[8];
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const float2 m = *reinterpret_cast<const float2 *>(smax + head(j));
                ref[j] = m.x;
                ref[j + 1] = m.y;
            }
            mbar_wait(bar_s + 8 * x, ph, abort_flag, p.status);
            after_sync();
            uint32_t s[2][8];
            tmem_ld_16x16(lane_base + kColS + 64 * x + hw, s[0]);
            tmem_ld_16x16(lane_base + kColS + 64 * x + hw + 16, s[1]);
            tmem_ld_wait();
            // logits in log2 units above the heads' references: v[r][j] of key row r, head j
            float v[2][8];
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[r][j] = kv[r] ? fmaf(__uint_as_float(s[j >> 2][4 * ((j >> 1) & 1) + 2 * r + (j & 1)]), c2, -ref[j]) : -INFINITY;
            float top = -INFINITY;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                top = fmaxf(top, fmaxf(v[0][j], v[1][j]));
            if (named_bar_or(slice_bar, 128, (fresh && (kv[0] || kv[1])) || top > kExceedLog2)) {
                // the block's maxima, by the four warps of these heads, become the references where they are larger
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float mx = fmaxf(v[0][j], v[1][j]);
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1)
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                    if (lane < 4)
                        red[quad * kNH + head(j)] = mx;
                }
                named_bar(slice_bar, 128);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int h = head(j);
                    const float m = fmaxf(fmaxf(red[h], red[kNH + h]), fmaxf(red[2 * kNH + h], red[3 * kNH + h]));
                    const float up = m == -INFINITY ? 0.f : fresh ? m : fmaxf(m, 0.f);   // (-inf: every logit is NaN)
                    const float fall = fresh ? 1.f : exp2_approx(-up);
                    l[j] *= fall;
                    v[0][j] -= up;
                    v[1][j] -= up;
                    if (quad == 0 && lane < 4) {
                        smax[h] += up;
                        fin[h] = fall;
                    }
                }
                named_bar(slice_bar, 128);   // the references and factors are written, and red is free again
                if (!fresh) {
                    // (b > 0: no key was seen before otherwise) P.V of block b - 1 has to be complete
                    mbar_wait(bar_pv + 32 * (x ^ 1) + 24, (uint32_t)((b - 1) >> 1) & 1u, abort_flag, p.status);
                    after_sync();
#pragma unroll 1
                    for (int m = 0; m < 8; ++m) {
                        const int hc = hw + 16 * (m & 1);
                        uint32_t y[16];
                        tmem_ld16(lane_base + kColO + 64 * (m >> 1) + hc, y);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            y[j] = __float_as_uint(__uint_as_float(y[j]) * fin[hc + j]);
                        tmem_st16(lane_base + kColO + 64 * (m >> 1) + hc, y);
                    }
                    tmem_st_wait();
                }
                fresh = false;
            }
            // P = 2^v -> BF16 P^T rows srow and srow + 8
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    const float p0 = exp2_approx(v[r][j]), p1 = exp2_approx(v[r][j + 1]);
                    l[j] += p0;
                    l[j + 1] += p1;
                    st_shared_u32(sK + (uint32_t)x * kKBytes + 8u * kChunkBytes + sw128(srow + 8 * r, (hw >> 3) + (j >> 1)) +
                                      4u * (lane & 3),
                                  pack_bf16x2(p0, p1));
                }
            fence_async_smem();
            before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar_p + 8 * x);
        }
        // row sums over the keys
#pragma unroll
        for (int j = 0; j < 8; ++j) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1)
                l[j] += __shfl_xor_sync(0xffffffffu, l[j], d);
            if (lane < 4)
                red[quad * kNH + head(j)] = l[j];
        }
        if (quad == 0)
            smax[hw + lane] = fresh ? -INFINITY : smax[hw + lane] * 0.6931471805599453f;
    }

    // ---- epilogue: the output's factors or the split's statistics, then the value tiles
    const int hs = 16 * (ww >> 2);   // workers: first of this warp's 16 heads
    if (warp >= 1 && warp <= kSoftmaxWarps) {
        named_bar(1, 32 * kSoftmaxWarps);
        if (tid - 32 < kNH) {
            const int h = tid - 32;
            const float lsum = (red[h] + red[kNH + h]) + (red[2 * kNH + h] + red[3 * kNH + h]);
            const float ms = smax[h];
            if (p.splits == 1) {
                const float sk = p.sink != nullptr && h < nhv ? p.sink[h0 + h] : -INFINITY;
                const float M = fmaxf(ms, sk);
                const float e = ms == -INFINITY ? 0.f : expf(ms - M);
                const float Z = (ms == -INFINITY ? 0.f : lsum * e) + (sk == -INFINITY ? 0.f : expf(sk - M));
                fin[h] = ms == -INFINITY ? 0.f : e / Z;
                if (p.lse != nullptr && h < nhv)
                    p.lse[(int64_t)t * p.num_heads + h0 + h] = M == -INFINITY ? -INFINITY : M + logf(Z);
            } else {
                fin[h] = lsum;
            }
        }
    }
    if (warp >= 1 && warp < kPvWarp)
        named_bar(4, 32 * (kSoftmaxWarps + kDequantWarps));
    if (is_worker) {
        mbar_wait(bar_pv + 32 * ((nblocks - 1) & 1) + 24, (uint32_t)((nblocks - 1) >> 1) & 1u, abort_flag, p.status);
        after_sync();
        if (p.splits == 1) {
#pragma unroll 1
            for (int m = 0; m < 4; ++m) {
                uint32_t y[16];
                tmem_ld16(lane_base + kColO + 64 * m + hs, y);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int h = hs + j;
                    if (h < nhv) {
                        const __nv_bfloat16 o = __float2bfloat16_rn(__uint_as_float(y[j]) * fin[h]);
                        p.out[((int64_t)t * p.num_heads + h0 + h) * kLatent + kDvTile * m + dv0] =
                            *reinterpret_cast<const uint16_t *>(&o);
                    }
                }
            }
        }
    }
    if (p.splits > 1) {
        // the split's partial goes from TMEM into the shared memory of each head's owner:
        // recv[split][head - owner's first head][512] in the owner's K tile region
        cluster_sync();   // every split is past its products: partials may land
        if (is_worker) {
            const int S = p.splits;
            const int hp = (kNH + S - 1) / S;
            if (wid < nhv)
                push_stat(smem_u32(gbase), S, split, wid, smax[wid], fin[wid]);
            const int r0 = hs / hp;   // this warp's 16 heads belong to owners r0, r0 + 1, r0 + 2 at most
#pragma unroll 1
            for (int m = 0; m < 4; ++m) {
                if (hs >= nhv)   // nhv is a multiple of 16: whole warps skip
                    break;
                uint32_t y[16];
                tmem_ld16(lane_base + kColO + 64 * m + hs, y);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int h = hs + j;
                    const int r = r0 + (h >= (r0 + 1) * hp) + (h >= (r0 + 2) * hp);
                    const uint32_t off = (uint32_t)(((split * hp + h - r * hp) * kLatent + kDvTile * m + dv0) * 4);
                    st_cluster_f32(map_to_rank(sK + off, (uint32_t)r), __uint_as_float(y[j]));
                }
            }
        }
    }
    before_sync();
    __syncthreads();
    after_sync();
    if (warp == 0)
        tmem_free(tmem, kTmemCols);
    if (p.splits > 1) {
        cluster_sync();   // every partial has landed
        merge_splits(p.out, p.lse, p.sink, p.num_heads, p.splits, t, h0, split,
                     reinterpret_cast<const float *>(gbase + kQBytes), reinterpret_cast<const float *>(gbase),
                     reinterpret_cast<float *>(gbase + 2048));
    }
}

}  // namespace

int decode_fp4_block_keys() { return kBK; }
int decode_fp4_max_splits() { return kMaxSplits; }

// Concurrently resident CTAs when launched in clusters of `splits` (whole clusters must fit inside one
// GPC); cached per device.
int decode_fp4_resident_ctas(int splits)
{
    static int cache[64][kMaxSplits + 1];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64 || splits < 1 || splits > kMaxSplits)
        return 0;
    if (cache[dev][splits] > 0)
        return cache[dev][splits];
    if (set_smem_once(reinterpret_cast<const void *>(decode_fp4_kernel), kSmemBytes, kAttrFp4) != cudaSuccess)
        return 0;
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    if (splits > 1) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(splits * n);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kSmemBytes;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = splits;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int clusters = 0;
        if (cudaOccupancyMaxActiveClusters(&clusters, reinterpret_cast<const void *>(decode_fp4_kernel), &cfg) != cudaSuccess) {
            cudaGetLastError();
            return 0;
        }
        n = clusters * splits;
    }
    cache[dev][splits] = n;
    return n;
}

cudaError_t launch_decode_fp4(const Decode4Params &p, cudaStream_t stream)
{
    if (p.num_tokens <= 0)
        return cudaSuccess;
    if (p.groups != (p.num_heads + kNH - 1) / kNH || p.splits < 1 || p.splits > kMaxSplits || p.chunk < 1)
        return cudaErrorInvalidValue;
    const cudaError_t e = set_smem_once(reinterpret_cast<const void *>(decode_fp4_kernel), kSmemBytes, kAttrFp4);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.num_tokens * (unsigned)p.groups * (unsigned)p.splits);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.splits;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.splits > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, decode_fp4_kernel, p);
}

}  // namespace dsv4
