// decode_fp4.cu -- sparse-MLA decode over the 4-bit cache on the tensor cores (tcgen05 / TMEM).
//
// Operation (per token t, head h, over the token's combined list of positions):
//   s_p = scale * q_h . k_p (576 dims),  lse_h = ln(sum_p e^{s_p} + e^{sink_h}),  out_h = sum_p e^{s_p - lse_h} v_p
// The lists of cache slots come from the list kernel (lists_fp4.cu) ahead of this one in the stream, or, with few units, are
// made here by the ten warps that do not bring Q (a launch less: 10.7 against 12.4 us for 2 tokens x 16 heads in a loop of
// calls).
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
// P.V of b runs.  (In one 128-key tile, whose steps form a chain, 128 tokens x 128 heads took 180 us where the first
// form with two tiles took 168.)
//   - a thread holds its eighth of a row's next entry in registers, loaded as those of the present block are
//     used up (two blocks ahead in registers: 140 against 135 us below; whole entries prefetched to L2: slower too);
//   - the softmax takes the logits of the unit's first key as references, and exchanges maxima between warps only
//     when a logit exceeds its head's reference by 40 (in log2 units): P and the sums are floating-point numbers,
//     whose relative precision does not depend on the reference, and 2^40 leaves fp32's sums of 2^24 keys room for
//     values up to 2^64 (those of normalised keys are about 1).
//     The usual block needs one barrier that ORs a predicate.  Row sums stay in registers.
//     Where few units are shared, the output is divided by the sum of the weights as rounded to BF16, so that a key that
//     has most of the weight loses nothing by its rounding (the lse keeps the exact sum; 1 % of the time of a small batch).
//
// What bounds it.  128 tokens x 128 heads x 2176 keys: 122 us in this kernel (131 with the lists and the join), 0.63 PFLOP/s,
// DRAM at 20 % of its peak, the tensor pipe busy 40 % of the time, issue slots 54 %.  A 64-key block takes 3.7 k cycles where
// the loop runs freely (4.1 k with the units' ends), and its steps are a chain over twice that, since its tile is one of two: the
// dequant 3.0 k to its last chunk, S^T 1.2 k after that, the softmax 1.7 k, P.V 1.4 k to the first chunks' release.  S^T of
// one block and P.V of the other meet and then take 116 of the 128 bytes a cycle of shared memory; letting either go first,
// or issuing both from one warp (a product takes it about 50 cycles), was slower: 140 and 159 us.  The dequant warps are
// busy for all of a block's time too, 1.4 k of it with conversion and stores and 1.1 k waiting for scale bytes and entries,
// so neither side alone is worth much: half of the dequant left out gives 127 us in all, no P.V 120, no gather 118.
//
// Work.  With up to half as many units as multiprocessors, as many CTAs as there are for it share each unit evenly.  Otherwise a
// persistent CTA per multiprocessor takes an equal run of the blocks of all units (the end of one unit,
// whole units, the start of another), so lists of any lengths fill the machine; with one unit per CTA, 256 equal
// units on 152 multiprocessors take two full waves.  26 warps: warp 0 issues S^T, warp 25 P.V, warps 1-8 do the
// softmax and the epilogue, warps 9-24 bring Q and the K tiles; the roles meet only at mbarriers, so the first blocks
// of a unit are dequantised while the last one's output is still written.  The parts of a unit that several CTAs share
// go to the workspace in fp32 and are joined by a kernel of their own.  16 or 32 heads run as a 64-head group
// whose missing heads have zero queries (their columns are computed and dropped).  Every mbarrier wait is bounded.
//
// Order of the dims inside a tile.  The eight 4-bit codes of a 32-bit word become the pairs (e_k, e_{k+4}):
// code k and code k + 4 lie 16 bits apart, so one shift puts both at their places in a BF16 pair (two masked
// shifts: magnitude and sign).  Inside each group of eight latent dims the tile therefore holds e0 e4 e1 e5 e2
// e6 e3 e7; Q is stored in the same order, and the epilogue writes each value dim to its own place.
#include <algorithm>
#include <climits>
#include <cuda_bf16.h>
#include <math.h>

#include "lists_fp4.cuh"
#include "tcgen05.cuh"

namespace dsv4 {
namespace {

using namespace tc;

constexpr int kSoftmaxWarps = 8;         // warps 1-8 (warp 0 issues S^T)
constexpr int kDequantWarp0 = 9;
constexpr int kDequantWarps = 16;        // warps 9-24: also Q's layout and the epilogue
constexpr int kPvWarp = 25;              // issues P.V
constexpr int kTmemWarp = 24;            // takes and frees the tensor memory (a warp that makes no list)
constexpr int kThreads = 832;
constexpr int kWorkers = 32 * kDequantWarps;
constexpr int kListThreads = kThreads - kWorkers;   // make a list while the others bring Q,
constexpr int kListLoads = 4;            // each with so many of its entries in flight: 1280 in all
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
constexpr int kJoinHeads = 4;            // heads per CTA of the joining kernel, a warp each
constexpr int kJoinSplit = 8;            // warps to a head where it may have kJoinMany parts or more
constexpr int kJoinMany = 8;
constexpr int kMinBlocks = 2;            // per CTA (with 1: 1 x 16 heads, 256 keys 11.8 -> 10.8 us, 16 x 64, 640 keys 16.7 -> 18.6)

// small shared region (after Q and the two K tiles)
constexpr int kOffRed = 0;               // float [4][64]: per-quadrant head maxima, or row sums at the end
constexpr int kOffMax = 1024;            // float [64]: reference maximum per head (log2 units; natural ones at the end)
constexpr int kOffFin = 1280;            // float [64]: the root of a rescale's factor; at the end the output's, or a split's row sum
constexpr int kOffValid = 1536;          // uint8 [2][64]: rows of a K tile that hold a key
constexpr int kOffBars = 1664;           // u64: bar_s[2], bar_p[2], bar_grp[2][2], bar_pv[2][4], bar_q, bar_o
constexpr int kOffTmem = 1808;           // u32
constexpr int kOffAbort = 1812;          // int
constexpr int kOffStart = 1816;          // int [8]: the unit at the run's start, its first block and the next unit's; at its end
constexpr int kOffScan = 1848;           // int [26]
constexpr int kOffRed2 = 1984;           // float [4][64]: the rounded weights' row sums at the end
constexpr int kSmallBytes = 3008;
constexpr int kSmemBytes = kQBytes + 2 * kKBytes + kSmallBytes + 1024;   // + alignment slack
constexpr int kQLoads = kNH * (kDim / 8) / kWorkers;                     // 9 16-byte Q pieces per worker
static_assert(kNH * (kDim / 8) % kWorkers == 0, "Q pieces per worker");
static_assert(2 * kKBytes >= 32768 + 4 * kListLoads * kListThreads / 32, "a list's sets fit the K tiles");
static_assert(16 * kListLoads * kListThreads <= 32768, "the rows of lists made here");
// a part in the workspace: O [64][512], then (m, l, l of the rounded weights, -) [64]
constexpr int kPartFloats = kNH * kLatent + 4 * kNH;

// instruction descriptors (kind::f16): D f32, A/B bf16, N = 64
constexpr uint32_t kIdescBase = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(kNH >> 3) << 17);
constexpr uint32_t kIdescQK = kIdescBase | ((uint32_t)(kBK >> 4) << 24);                              // A, B K-major
constexpr uint32_t kIdescPV = kIdescBase | ((uint32_t)(kDvTile >> 4) << 24) | (1u << 15) | (1u << 16);   // A, B MN-major

// 16 bytes of an entry.  Entries start at odd multiples of 16 bytes as often as at even ones, so a row's 64-byte
// pieces share 32-byte sectors with their neighbours: L1 keeps them for the next piece (8 % of the kernel's time
// against loads that do not allocate there).
__device__ __forceinline__ uint4 ld16(const void *p) { return __ldca(reinterpret_cast<const uint4 *>(p)); }

// 32 E2M1 codes times 2^(se - 127) -> 32 BF16 values, exactly, into the four 16-byte units u .. u + 3 (xored with x)
// of the row at shared address rb.
// A code's exponent and mantissa bits at the low end of the BF16 exponent are its value times 2^-126 (both
// formats put the binary point the same way, subnormals included); one multiply by 2^(se - 1) gives the value.
// Scales past 2 (se > 128, whose factor has no BF16 form) take a second multiply, 255 (NaN) among them.
__device__ __forceinline__ void dequant32_store(const uint4 &v, uint32_t se, uint32_t rb, uint32_t u, uint32_t x)
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

// The work of this CTA.  A unit is a (token, 64-head group), in the order of groups and then tokens (CTAs that take the
// groups of one token then run at about the same time and find its entries in L2); blocks are counted over all units.
// Every role of the CTA walks the same blocks.
struct Walk {
    int w, w1;        // blocks [w, w1) are still to do
    int t, h0;        // token and first head of the unit of block w
    int start;        // that unit's first block
    int len;          // its keys
};

struct Segment {
    int t, h0;
    int kb, nb;       // blocks kb .. kb + nb - 1 of the unit
    int len;          // the unit's keys
};

__device__ __forceinline__ int blocks_of(int len) { return (len + kBK - 1) / kBK; }

__device__ __forceinline__ bool next_segment(Walk &k, const Decode4Params &p, Segment &s)
{
    if (k.w >= k.w1)
        return false;
    int blocks;
    while (true) {   // (units without keys have no block)
        blocks = blocks_of(k.len);
        if (k.start + blocks > k.w)
            break;
        k.start += blocks;
        if (++k.t == p.num_tokens) {
            k.t = 0;
            k.h0 += kNH;
        }
        k.len = __ldcg(p.lens + k.t);
    }
    s.len = k.len;
    s.t = k.t;
    s.h0 = k.h0;
    s.kb = k.w - k.start;
    s.nb = min(blocks - s.kb, k.w1 - k.w);
    k.w += s.nb;
    return true;
}

// first block of CTA c's run, and the CTA whose run holds block w (G runs over all W blocks)
__device__ __forceinline__ int run_start(int c, int W, int G)   // floor(c W / G)
{
    const unsigned q = (unsigned)W / (unsigned)G, r = (unsigned)W % (unsigned)G;
    return (int)(q * (unsigned)c + r * (unsigned)c / (unsigned)G);
}

__device__ __forceinline__ int run_of(int w, int W, int G) { return (int)(((long long)(w + 1) * G - 1) / W); }

// The queries of 64 heads -> swizzled K-major B operand, in the tile's order of dims (zeros for heads that do not
// exist), by worker wid of 512, kBatch pieces in flight.
template <int kBatch>
__device__ __forceinline__ void store_q(const Decode4Params &p, int t, int h0, uint32_t sQ, int wid)
{
    const uint4 *q = reinterpret_cast<const uint4 *>(p.q + (int64_t)t * p.q_token_stride + h0 * kDim);
    const int pieces = min(kNH, p.num_heads - h0) * (kDim / 8);
#pragma unroll 1
    for (int j0 = 0; j0 < kQLoads; j0 += kBatch) {
        uint4 v[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int i = wid + kWorkers * (j0 + j);
            v[j] = i < pieces ? __ldca(q + i) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int i = wid + kWorkers * (j0 + j);
            const int h = i / (kDim / 8), c = i % (kDim / 8);
            const uint32_t a = sQ + (c >> 3) * kQChunkBytes + sw128(h, c & 7);
            if (c < kLatent / 8)
                st_shared_v4(a, __byte_perm(v[j].x, v[j].z, 0x5410), __byte_perm(v[j].x, v[j].z, 0x7632),
                             __byte_perm(v[j].y, v[j].w, 0x5410), __byte_perm(v[j].y, v[j].w, 0x7632));
            else
                st_shared_v4(a, v[j].x, v[j].y, v[j].z, v[j].w);
        }
    }
}

// O^T from TMEM to the output (times the heads' factors) or to a part of it, 16 heads of a value tile at a time, by
// warp `rank` of the `warps` that share the quadrant.
__device__ __forceinline__ void write_o(const Decode4Params &p, int t, int h0, float *part, const float *fin,
                                        uint32_t lane_base, int quad, int lane, int rank, int warps)
{
    const int slices = min(kNH, p.num_heads - h0) / 16;   // (heads that exist: a multiple of 16)
    const int vrow = quad * 32 + lane;                    // this lane's row of a value tile,
    const int dv0 = (vrow & ~7) | ((vrow >> 1) & 3) | ((vrow & 1) << 2);   // and its value dim (the tile's order of dims)
#pragma unroll 1
    for (int i = rank; i < 4 * slices; i += warps) {
        const int m = i / slices, hc = 16 * (i % slices), dv = kDvTile * m + dv0;
        uint32_t y[16];
        tmem_ld16(lane_base + kColO + 64 * m + hc, y);
        tmem_ld_wait();
        if (part == nullptr) {
            uint16_t *o = p.out + ((int64_t)t * p.num_heads + h0 + hc) * kLatent + dv;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const __nv_bfloat16 v = __float2bfloat16_rn(__uint_as_float(y[j]) * fin[hc + j]);
                o[j * kLatent] = *reinterpret_cast<const uint16_t *>(&v);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                __stcg(part + (hc + j) * kLatent + dv, __uint_as_float(y[j]));
        }
    }
}

struct SyncLists {   // the threads that make a list
    __device__ __forceinline__ void operator()() const { named_bar(5, kListThreads); }
    __device__ __forceinline__ bool any(bool v) const { return named_bar_or(5, kListThreads, v); }
};

// CTAs that share a unit of W blocks evenly
__device__ __forceinline__ int shares_of(const Decode4Params &p, int W)
{
    return max(1, min(p.ctas_per_unit, (W + kMinBlocks - 1) / kMinBlocks));
}

// kShared: few units, each shared evenly by p.ctas_per_unit CTAs, which make its token's list themselves (p.own_lists) unless
// the rows are wide; otherwise every CTA takes an equal run of the blocks of all units.  (In one kernel the second kind took
// 2 % longer: registers.)
template <bool kShared>
__global__ void __launch_bounds__(kThreads, 1) decode_fp4_kernel(const Decode4Params p)
{
    extern __shared__ uint8_t smem_raw[];
    const int tid = threadIdx.x;
    const int warp = tid >> 5;
    const int lane = tid & 31;
    const bool is_worker = warp >= kDequantWarp0 && warp < kDequantWarp0 + kDequantWarps;

    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;   // the swizzled tiles start on 1024-byte boundaries
    uint8_t *gbase = smem_raw + (base - raw);
    const uint32_t sQ = base;
    const uint32_t sK = base + kQBytes;           // two K tiles; P^T takes a tile's rope chunk once its S^T is done
    uint8_t *small = gbase + kQBytes + 2 * kKBytes;
    float *red = reinterpret_cast<float *>(small + kOffRed);
    float *red2 = reinterpret_cast<float *>(small + kOffRed2);
    float *smax = reinterpret_cast<float *>(small + kOffMax);
    float *fin = reinterpret_cast<float *>(small + kOffFin);
    uint8_t *valid = small + kOffValid;
    const uint32_t bar_s = smem_u32(small + kOffBars);   // [tile] S^T complete
    const uint32_t bar_p = bar_s + 16;                   // [tile] P^T written (softmax warps)
    const uint32_t bar_grp = bar_s + 32;                 // [tile][2] column chunks 0-3, then 4-8 written (dequant warps)
    const uint32_t bar_pv = bar_s + 64;                  // [tile][4] P.V of value tile m complete
    const uint32_t bar_q = bar_s + 128;                  // Q of the segment written (dequant warps)
    const uint32_t bar_o = bar_s + 136;                  // O^T of the segment read (softmax warps)
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(small + kOffTmem);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(small + kOffAbort);
    int *first = reinterpret_cast<int *>(small + kOffStart);
    int *scan = reinterpret_cast<int *>(small + kOffScan);

    // ---- set-up that reads no list
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar_s + 8 * i, 1);
            mbar_init(bar_p + 8 * i, kSoftmaxWarps);
        }
        for (int i = 0; i < 4; ++i)
            mbar_init(bar_grp + 8 * i, kDequantWarps);
        for (int i = 0; i < 8; ++i)
            mbar_init(bar_pv + 8 * i, 1);
        mbar_init(bar_q, kDequantWarps);
        mbar_init(bar_o, kSoftmaxWarps);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        *abort_flag = 0;
    }
    // (tensor memory is taken when no kernel but this library's own list kernel can still be running ahead of this one)
    const bool own_lists = kShared && p.own_lists;
    if (own_lists)
        griddep_wait();
    if (warp == kTmemWarp)
        tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    // ---- this CTA's blocks
    Walk walk;
    int W = 0, G = 1, w0 = 0;
    if constexpr (kShared) {   // an equal share of one unit
        const int unit = blockIdx.x / p.ctas_per_unit, s = blockIdx.x % p.ctas_per_unit;
        walk.t = unit % p.num_tokens;
        walk.h0 = unit / p.num_tokens * kNH;
        walk.start = 0;
        if (is_worker) {
            // (where a list kernel is ahead, it let this one begin after everything before it in the stream had ended: the
            // queries are there, and come in while the lists are made)
            store_q<kQLoads>(p, walk.t, walk.h0, sQ, tid - 32 * kDequantWarp0);
        } else if (own_lists) {
            const int ltid = warp < kDequantWarp0 ? tid : tid - kWorkers;
            // Every CTA of a token writes the slots of its top-k entries, the same ones to the same places, and those of the
            // window's part that it needs.
            uint8_t *tab = gbase + kQBytes;   // (the K tiles' place)
            const int len = lists::build<kListThreads, kListLoads>(
                p.lists, walk.t, ltid, reinterpret_cast<unsigned long long *>(tab),
                reinterpret_cast<int *>(tab + p.lists.smem_bytes), SyncLists(), [&](int n) {
                    const int blocks = blocks_of(n), g = shares_of(p, blocks);
                    return s < g ? make_int2(run_start(s, blocks, g) * kBK, run_start(s + 1, blocks, g) * kBK) : make_int2(n, n);
                });
            if (ltid == 0)
                first[0] = len;
        }
        if (!own_lists)
            griddep_wait();
        before_sync();
        __syncthreads();
        walk.len = own_lists ? first[0] : __ldcg(p.lens + walk.t);
        W = blocks_of(walk.len);
        G = shares_of(p, W);
        walk.w = s < G ? run_start(s, W, G) : W;
        walk.w1 = s < G ? run_start(s + 1, W, G) : W;
        if (own_lists && s == 0 && G == 1 && tid == 0)
            p.joins[unit] = make_int2(0, 0);
        if (own_lists && s == 0 && W == 0) {   // a token without a key
            const int nhv = min(kNH, p.num_heads - walk.h0);
            const int64_t row = (int64_t)walk.t * p.num_heads + walk.h0;
            for (int i = tid; i < nhv * kLatent / 8; i += kThreads)
                *reinterpret_cast<uint4 *>(p.out + row * kLatent + 8 * i) = make_uint4(0, 0, 0, 0);
            if (p.lse != nullptr && tid < nhv)
                p.lse[row + tid] = p.sink != nullptr ? p.sink[walk.h0 + tid] : -INFINITY;
        }
    } else {                     // an equal run of the blocks of all units
        griddep_wait();
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
        int excl = incl - mine, all = 0;   // of one group
        for (int i = 0; i < kThreads / 32; ++i) {
            excl += i < warp ? scan[i] : 0;
            all += scan[i];
        }
        W = all * p.groups;
        G = max(1, min((int)gridDim.x, (W + kMinBlocks - 1) / kMinBlocks));
        walk.w = blockIdx.x < G ? run_start(blockIdx.x, W, G) : W;
        walk.w1 = blockIdx.x < G ? run_start(blockIdx.x + 1, W, G) : W;
        // the unit that holds block w: token, group, first block, and the next unit's
        auto find = [&](int w, int *out) {
            const int r = all > 0 ? w % all : 0;
            if (w < W && mine > 0 && excl <= r && r < excl + mine) {
                int at = excl, t = t0, n;
                while (at + (n = blocks_of(__ldcg(p.lens + t))) <= r) {
                    at += n;
                    ++t;
                }
                out[0] = t;
                out[1] = w / all * kNH;
                out[2] = w - r + at;
                out[3] = out[2] + n;
            }
        };
        find(walk.w, first);
        if (!p.split)
            find(walk.w1, first + 4);
        before_sync();
        __syncthreads();
        walk.t = first[0];
        walk.h0 = first[1];
        walk.start = first[2];
        walk.len = walk.w < walk.w1 ? __ldcg(p.lens + walk.t) : 0;
        if (!p.split) {   // a run begins and ends at the next start of a unit
            if (walk.w < W && walk.w > first[2])
                walk.w = first[3];
            if (walk.w1 < W)
                walk.w1 = walk.w1 > first[6] ? first[7] : first[6];
        }
        w0 = walk.w;
    }
    __syncthreads();   // barriers, TMEM address
    after_sync();
    const uint32_t tmem = *tmem_slot;

    griddep_launch();   // (the joining kernel waits for this grid itself)
    const int quad = warp & 3;                            // TMEM lane quadrant of this warp
    const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
    Segment seg;

    if (warp == 0) {
        // descriptors: K-major operands advance 32 B per 16 dims and one column chunk per 64
        const uint32_t leader = elect_one();
        const uint64_t qk_a = sdesc(sK, 16, 1024);
        const uint64_t qk_b = sdesc(sQ, 16, 1024);
        uint32_t g = 0;   // blocks since the kernel began: tile g & 1, phase g >> 1
        for (uint32_t n = 0; next_segment(walk, p, seg); ++n) {
            mbar_wait(bar_q, n & 1u, abort_flag, p.status);
            for (int b = 0; b < seg.nb; ++b, ++g) {
                const uint32_t x = g & 1u, ph = (g >> 1) & 1u;
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
        }
    } else if (warp == kPvWarp) {
        // MN-major operands advance 2 KB per 16 keys
        const uint32_t leader = elect_one();
        const uint64_t pv_a = sdesc(sK, kChunkBytes, 1024);
        const uint64_t pv_b = sdesc(sK + 8 * kChunkBytes, 1024, 1024);
        uint32_t g = 0;
        for (uint32_t n = 0; next_segment(walk, p, seg); ++n) {
            if (n > 0) {
                mbar_wait(bar_o, (n - 1) & 1u, abort_flag, p.status);   // the last segment's O^T has been read
                after_sync();
            }
            for (int b = 0; b < seg.nb; ++b, ++g) {
                const uint32_t x = g & 1u;
                mbar_wait(bar_p + 8 * x, (g >> 1) & 1u, abort_flag, p.status);
                after_sync();
                const uint64_t off = (uint64_t)((x * kKBytes) >> 4);
                const int left = seg.len - (seg.kb + b) * kBK;   // 16-key steps without a key are left out
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
        }
    } else if (is_worker) {
        // ---- Q's layout, and the dequant: eight threads to a row, each with two 16-byte pieces of codes (32 dims each),
        // one of rope and two scale bytes.  A warp takes four rows whose numbers differ mod 4: eight lanes that store
        // together (four rows, an even and an odd piece) meet eight different bank groups, and a load covers 128
        // contiguous bytes of a row (against eight rows of 64 bytes: 4 % of the kernel's time).  The rows spread over the
        // tile, so that a short block keeps every warp at work.
        const int ww = warp - kDequantWarp0;
        const int wid = 32 * ww + lane;
        const int piece = 2 * (lane >> 3) + ((lane >> 2) & 1), runit = 4 * ((lane >> 2) & 1) + (lane >> 3);
        const int rrow = 8 * (((ww >> 1) - (lane & 3)) & 7) + 4 * (ww & 1) + (lane & 3);
        const uint32_t rb = (uint32_t)(rrow >> 3) * 1024u + (uint32_t)(rrow & 7) * 128u;
        const uint32_t x7 = (uint32_t)(rrow & 7);
        uint32_t g = 0;
        for (uint32_t n = 0; next_segment(walk, p, seg); ++n) {
            const int t = seg.t, h0 = seg.h0;
            const int32_t *list = p.slots + (int64_t)t * p.list_w;
            // Cache slots (-1 past the list's end): a lane holds that of its row (lane % 4) in block lane / 4 of eight, so
            // that one load in eight blocks, and no wait for it among the entries' loads, feeds the warp.
            auto load_slots = [&](int b8) {
                const int b = b8 + (lane >> 2), i = (seg.kb + b) * kBK + rrow;
                return b < seg.nb && i < seg.len ? __ldcg(list + i) : -1;
            };
            int slots = load_slots(0), slots_next = load_slots(8);
            auto slot_of = [&](int b) { return __shfl_sync(0xffffffffu, slots, 4 * (b & 7) + (lane & 3)); };
            auto entry = [&](int slot) { return p.kv + (int64_t)(slot >= 0 ? slot : 0) * kEntry4Bytes; };
            // the entry of the block ahead; lanes 4 i .. 4 i + 3 (i < 4) hold word i of the rows' scale bytes
            uint4 pre[2], prope;
            uint32_t psc = 0u;
            auto load_piece = [&](const uint8_t *e, int m) { pre[m] = ld16(e + 128 * m + 16 * piece); };
            auto load_scales = [&](const uint8_t *e) {
                if (lane < 16)
                    psc = __ldca(reinterpret_cast<const uint32_t *>(e + kScale4Offset) + (lane >> 2));
            };
            const int slot0 = slot_of(0);
            bool pre_ok = slot0 >= 0;
            if (pre_ok) {
                load_piece(entry(slot0), 0);
                load_piece(entry(slot0), 1);
                load_scales(entry(slot0));
                prope = ld16(entry(slot0) + kRope4Offset + 16 * runit);
            }
            if (n > 0 || !kShared) {
                if (n > 0)   // S^T of the last segment's last block is done with its Q
                    mbar_wait(bar_s + 8 * ((g - 1) & 1u), ((g - 1) >> 1) & 1u, abort_flag, p.status);
                store_q<3>(p, t, h0, sQ, wid);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar_q);

            for (int b = 0; b < seg.nb; ++b, ++g) {   // a block into its K tile (zeros for rows without a key)
                const uint32_t x = g & 1u, ph = ((g >> 1) - 1) & 1u;
                const uint32_t tile = sK + x * kKBytes + rb;
                if ((b & 7) == 7) {
                    slots = slots_next;
                    slots_next = load_slots(b + 9);
                }
                const int slot1 = slot_of(b + 1);
                const bool ok_next = slot1 >= 0;
                const uint8_t *en = entry(slot1);   // the next block's entry goes into the registers as they are used up
                uint32_t se[2];   // the scales of this lane's pieces
#pragma unroll
                for (int m = 0; m < 2; ++m)
                    se[m] = (__shfl_sync(0xffffffffu, psc, 4 * (2 * m + (piece >> 2)) + (lane & 3)) >> (8 * (piece & 3))) & 0xFFu;
                if (ok_next)
                    load_scales(en);
#pragma unroll
                for (int m = 0; m < 2; ++m) {   // dims 256 m + 32 piece ..
                    if (g >= 2)   // P.V of the block before the last is done with these chunks
                        mbar_wait(bar_pv + 32 * x + 16 * m + 8, ph, abort_flag, p.status);
                    if (m == 0 && piece == 0)
                        valid[x * kBK + rrow] = pre_ok;
                    const uint32_t cb = tile + (uint32_t)(4 * m + (piece >> 1)) * kChunkBytes;
                    const uint32_t u = 4u * (uint32_t)(piece & 1);
                    if (pre_ok) {
                        dequant32_store(pre[m], se[m], cb, u, x7);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            st_shared_v4(cb + (((u + i) ^ x7) << 4), 0u, 0u, 0u, 0u);
                    }
                    if (ok_next)
                        load_piece(en, m);
                    if (m == 1) {   // the rope chunk, whose place P^T had
                        if (!pre_ok)
                            prope = make_uint4(0u, 0u, 0u, 0u);
                        st_shared_v4(tile + 8u * kChunkBytes + (((uint32_t)runit ^ x7) << 4), prope.x, prope.y, prope.z, prope.w);
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(bar_grp + 16 * x + 8 * m);
                }
                if (ok_next)
                    prope = ld16(en + kRope4Offset + 16 * runit);
                pre_ok = ok_next;
            }
            if (kShared) {   // the CTA's only segment: its output is written by all
                named_bar(4, 32 * kSoftmaxWarps + kWorkers);   // (the factors are there)
                mbar_wait(bar_pv + 32 * ((g - 1) & 1u) + 24, ((g - 1) >> 1) & 1u, abort_flag, p.status);
                after_sync();
                write_o(p, t, h0, seg.nb == blocks_of(seg.len) ? nullptr : p.parts + (size_t)(2 * blockIdx.x) * kPartFloats,
                        fin, lane_base, quad, lane, 2 + (ww >> 2), 6);
            }
        }
    } else {
        // ---- softmax and epilogue
        constexpr int kAll = 32 * kSoftmaxWarps;
        const int wid = tid - 32;
        const float c2 = p.scale * 1.4426950408889634f;   // logits in log2 units per raw dot product
        const int hw = 32 * ((warp - 1) >> 2);            // first of this warp's 32 heads; its 16 keys are the quadrant's
        const int slice_bar = 2 + ((warp - 1) >> 2);      // the four warps of these heads
        // this lane's keys are srow and srow + 8; its heads, j = 0..7:
        const int srow = 16 * quad + (lane >> 2);
        const int sh = hw + 2 * (lane & 3);
        auto head = [&](int j) { return sh + 16 * (j >> 2) + 8 * ((j >> 1) & 1) + (j & 1); };
        uint32_t g = 0;
        while (next_segment(walk, p, seg)) {
            const int t = seg.t, h0 = seg.h0;
            const int nhv = min(kNH, p.num_heads - h0);
            if (quad == 0)
                smax[hw + lane] = 0.f;
            named_bar(slice_bar, 128);
            float l[8];                                       // row sums of those heads over this lane's keys
#pragma unroll
            for (int j = 0; j < 8; ++j)
                l[j] = 0.f;
            float lr[kShared ? 8 : 1];                        // the same of the weights as P.V takes them, rounded to BF16
#pragma unroll
            for (int j = 0; j < (kShared ? 8 : 0); ++j)
                lr[j] = 0.f;
            uint32_t unset = 0xFFu;                           // bit j: head j has no reference (no logit above -inf so far)

            for (int b = 0; b < seg.nb; ++b, ++g) {
                const uint32_t x = g & 1u, ph = (g >> 1) & 1u;
                mbar_wait(bar_grp + 16 * x, ph, abort_flag, p.status);   // (complete by then: the rows' flags are visible)
                const bool kv[2] = {valid[x * kBK + srow] != 0, valid[x * kBK + srow + 8] != 0};   // (not past the list's end)
                float ref[8];
#pragma unroll
                for (int j = 0; j < 8; j += 2) {   // (in the first block they are 0, and may be being set)
                    const float2 m = b > 0 ? *reinterpret_cast<const float2 *>(smax + head(j)) : make_float2(0.f, 0.f);
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
                        v[r][j] = fmaf(__uint_as_float(s[j >> 2][4 * ((j >> 1) & 1) + 2 * r + (j & 1)]), c2, -ref[j]);
                if (!__all_sync(0xffffffffu, kv[0] && kv[1])) {   // (few blocks have rows without a key: 132.5 -> 131.6 us)
#pragma unroll
                    for (int r = 0; r < 2; ++r)
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            v[r][j] = kv[r] ? v[r][j] : -INFINITY;
                }
                if (b == 0 && valid[x * kBK] != 0) {
                    // any finite logit will do as a reference: those of the segment's first key
                    if (srow == 0) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            smax[head(j)] = v[0][j];
                    }
                    named_bar(slice_bar, 128);
                    unset = 0u;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float m = smax[head(j)];
                        const bool ok = fabsf(m) < INFINITY;
                        v[0][j] -= ok ? m : 0.f;
                        v[1][j] -= ok ? m : 0.f;
                        unset |= ok ? 0u : 1u << j;   // (this block's maxima replace it below)
                    }
                }
                float top = -INFINITY;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    top = fmaxf(top, fmaxf(v[0][j], v[1][j]));
                if (named_bar_or(slice_bar, 128, (unset != 0u && (kv[0] || kv[1])) || top > kExceedLog2)) {
                    // the block's maxima, by the four warps of these heads, become the references where they are larger or
                    // there is none (logits below 2^-126 of one that is too high would vanish, all of a head's among them)
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
                        const bool none = (unset >> j) & 1u;
                        const float up = m == -INFINITY ? 0.f : none ? m : fmaxf(m, 0.f);   // (-inf: every logit is that or NaN)
                        // (half of the fall, taken twice: what it is taken from may be 2^40 and more, so that the whole of
                        // it, below 2^-126, would lose weights that are not)
                        const float fall = none ? 1.f : exp2_approx(-0.5f * up);
                        unset &= m == -INFINITY ? ~0u : ~(1u << j);
                        l[j] = l[j] * fall * fall;
                        if constexpr (kShared)
                            lr[j] = lr[j] * fall * fall;
                        v[0][j] -= up;
                        v[1][j] -= up;
                        if (quad == 0 && lane < 4) {
                            smax[h] = none ? up : smax[h] + up;
                            fin[h] = fall;
                        }
                    }
                    named_bar(slice_bar, 128);   // the references and factors are written, and red is free again
                    if (b > 0) {   // O^T holds something: P.V of the block before has to be complete
                        mbar_wait(bar_pv + 32 * (x ^ 1u) + 24, ((g - 1) >> 1) & 1u, abort_flag, p.status);
                        after_sync();
#pragma unroll 1
                        for (int m = 0; m < 8; ++m) {
                            const int hc = hw + 16 * (m & 1);
                            uint32_t y[16];
                            tmem_ld16(lane_base + kColO + 64 * (m >> 1) + hc, y);
                            tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                y[j] = __float_as_uint(__uint_as_float(y[j]) * fin[hc + j] * fin[hc + j]);
                            tmem_st16(lane_base + kColO + 64 * (m >> 1) + hc, y);
                        }
                        tmem_st_wait();
                    }
                }
                // P = 2^v -> BF16 P^T rows srow and srow + 8
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int j = 0; j < 8; j += 2) {
                        const float p0 = exp2_approx(v[r][j]), p1 = exp2_approx(v[r][j + 1]);
                        l[j] += p0;
                        l[j + 1] += p1;
                        const uint32_t pk = pack_bf16x2(p0, p1);
                        if constexpr (kShared) {
                            lr[j] += __uint_as_float(pk << 16);
                            lr[j + 1] += __uint_as_float(pk & 0xFFFF0000u);
                        }
                        st_shared_u32(sK + x * kKBytes + 8u * kChunkBytes + sw128(srow + 8 * r, (hw >> 3) + (j >> 1)) +
                                          4u * (lane & 3),
                                      pk);
                    }
                fence_async_smem();
                before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar_p + 8 * x);
            }

            // ---- the segment's row sums and references (natural-log units)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1)
                    l[j] += __shfl_xor_sync(0xffffffffu, l[j], d);
                if (lane < 4)
                    red[quad * kNH + head(j)] = l[j];
                if constexpr (kShared) {
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1)
                        lr[j] += __shfl_xor_sync(0xffffffffu, lr[j], d);
                    if (lane < 4)
                        red2[quad * kNH + head(j)] = lr[j];
                }
            }
            if (quad == 0)
                smax[hw + lane] *= 0.6931471805599453f;
            named_bar(1, kAll);
            const bool whole = seg.nb == blocks_of(seg.len);
            float *part = nullptr;   // this CTA's part of a split unit
            if (!whole) {
                const int slot = walk.start > w0 ? 1 : 0;   // (the unit begins in this run, or with it or before it)
                part = p.parts + (size_t)(2 * blockIdx.x + slot) * kPartFloats;
                if (seg.kb == 0 && wid == 0) {   // its first part says how many there are, and which
                    const int n = kShared ? G : run_of(walk.start + blocks_of(seg.len) - 1, W, G) - (int)blockIdx.x + 1;
                    p.joins[h0 / kNH * p.num_tokens + t] = make_int2(2 * blockIdx.x + slot, n);
                }
            }
            if (wid < kNH) {
                const int h = wid;
                const float lsum = (red[h] + red[kNH + h]) + (red[2 * kNH + h] + red[3 * kNH + h]);
                const float lround = kShared ? (red2[h] + red2[kNH + h]) + (red2[2 * kNH + h] + red2[3 * kNH + h]) : lsum;
                // (no key, or logits of -inf alone: as a segment without keys.  With a reference that some logit has, or had
                // and was raised to another's, the sum is about 1 or more)
                const float ms = lsum == 0.f ? -INFINITY : smax[h];
                if (whole) {
                    const float sk = p.sink != nullptr && h < nhv ? p.sink[h0 + h] : -INFINITY;
                    const float M = fmaxf(ms, sk);
                    const float e = ms == -INFINITY ? 0.f : expf(ms - M);
                    const float zs = sk == -INFINITY ? 0.f : sk == M ? 1.f : expf(sk - M);   // (a sink of +inf takes all)
                    const float Z = (ms == -INFINITY ? 0.f : lsum * e) + zs;
                    fin[h] = ms == -INFINITY ? 0.f : e / (kShared ? lround * e + zs : Z);
                    if (p.lse != nullptr && h < nhv)
                        p.lse[(int64_t)t * p.num_heads + h0 + h] = M == -INFINITY ? -INFINITY : M + logf(Z);
                } else {
                    *reinterpret_cast<float4 *>(part + kNH * kLatent + 4 * h) =
                        ms == -INFINITY ? make_float4(ms, 0.f, 0.f, 0.f) : make_float4(ms, lsum, lround, 0.f);
                }
            }
            named_bar(1, kAll);
            mbar_wait(bar_pv + 32 * ((g - 1) & 1u) + 24, ((g - 1) >> 1) & 1u, abort_flag, p.status);
            after_sync();
            // ---- O^T out of TMEM (alone: two warps to a quadrant; with the dequant's six)
            if (kShared) {
                named_bar(4, kAll + kWorkers);
                write_o(p, t, h0, whole ? nullptr : part, fin, lane_base, quad, lane, (warp - 1) >> 2, 6);
            } else {
                write_o(p, t, h0, whole ? nullptr : part, fin, lane_base, quad, lane, (warp - 1) >> 2, 2);
            }
            before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar_o);
            named_bar(1, kAll);   // red, smax and fin are free again
        }
    }
    before_sync();
    __syncthreads();
    after_sync();
    if (warp == kTmemWarp)
        tmem_free(tmem, kTmemCols);
}

// e^x times sums that may be 2^40 and more: where it is small (x is the same in a warp) half of it goes into them first, since
// by itself it could go below 2^-126 and lose weights that fp32 holds.  Returns what is left to multiply by.
template <int kVecs>
__device__ __forceinline__ float exp_of(float x, float &z, float &zr, float4 (&o)[kVecs])
{
    if (x < -60.f) {
        x *= 0.5f;
        const float h = expf(x);
        z *= h;
        zr *= h;
#pragma unroll
        for (int k = 0; k < kVecs; ++k)
            o[k] = make_float4(o[k].x * h, o[k].y * h, o[k].z * h, o[k].w * h);
    }
    return expf(x);
}

// Joins the parts of the units that several CTAs shared, in the order of the parts:
//   m = max(max_c m_c, sink), Z = sum_c l_c e^{m_c - m} + e^{sink - m},
//   out = sum_c e^{m_c - m} O_c / Z  (BF16),  lse = m + ln Z
// A warp to a head, or kSplit of them, each with a run of the parts, where there may be many (one token x 16 heads over 131072
// keys, 152 parts: 81 us in all with one warp, 45.5 with eight; 17 parts: 16.8 and 15.0; four parts: 20.6 and 24.8).  The parts
// come from L2, kJoinBatch at a time with every load in flight: four where few CTAs share each unit (latency is all there is; they
// are read before it is known how many of them had work), two where runs of blocks end inside units (two parts are usual, and more registers would leave fewer warps: 8
// against 10.5 us for 151 split units).  (Joined inside the decode, by the CTA of a unit that finished last, the 256
// threads that are free there hold too few bytes in flight: a unit took 25 us.)
template <int kJoinBatch, int kSplit, bool kShared>
__global__ void __launch_bounds__(kSplit == 1 ? 32 * kJoinHeads : 32 * kSplit) join_parts_kernel(const Decode4Params p)
{
    const int unit = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = unit % p.num_tokens, h0 = unit / p.num_tokens * kNH;
    const int h = kSplit == 1 ? kJoinHeads * blockIdx.y + warp : blockIdx.y;   // head of the group
    griddep_wait();
    const int2 join = __ldcg(p.joins + unit);   // (slot of the first part, parts); zeros for a unit of one part
    int first = 2 * unit * p.ctas_per_unit, most = p.ctas_per_unit;
    if (p.ctas_per_unit == 0) {
        first = join.x;
        most = join.y;
    }
    const int share = (most + kSplit - 1) / kSplit, lo = kSplit == 1 ? 0 : warp * share, hi = min(most, lo + share);
    const float sk = p.sink != nullptr && (kSplit == 1 || warp == 0) ? p.sink[h0 + h] : -INFINITY;
    float M = sk, Z = sk == -INFINITY ? 0.f : 1.f, Zr = Z;   // (Zr: with the weights as rounded)
    float4 acc[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c0 = lo; c0 < hi; c0 += kJoinBatch) {
        float2 ml[kJoinBatch];
        float lr[kJoinBatch] = {};
        float4 o[kJoinBatch][4];
#pragma unroll
        for (int c = 0; c < kJoinBatch; ++c) {
            // the first part may be its CTA's second; the others are their CTAs' first
            const float *pc = p.parts + (size_t)(c0 + c == 0 ? first : 2 * (first / 2 + c0 + c)) * kPartFloats;
            if (c0 + c < hi) {
                ml[c] = __ldcg(reinterpret_cast<const float2 *>(pc + kNH * kLatent + 4 * h));
                if (kShared)
                    lr[c] = __ldcg(pc + kNH * kLatent + 4 * h + 2);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    o[c][k] = __ldcg(reinterpret_cast<const float4 *>(pc + h * kLatent + 128 * k + 4 * lane));
            }
        }
        if (c0 >= join.y)
            break;
        float m = M;
#pragma unroll
        for (int c = 0; c < kJoinBatch; ++c) {
            if (c0 + c >= min(hi, join.y))
                ml[c] = make_float2(-INFINITY, 0.f);
            m = fmaxf(m, ml[c].x);
        }
        // (both may be a sink of +inf, or -inf while all sums are 0)
        const float fall = M == m ? 1.f : exp_of(M - m, Z, Zr, acc);
        Z *= fall;
        if (kShared)
            Zr *= fall;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            acc[k].x *= fall;
            acc[k].y *= fall;
            acc[k].z *= fall;
            acc[k].w *= fall;
        }
#pragma unroll
        for (int c = 0; c < kJoinBatch; ++c) {
            if (ml[c].x == -INFINITY)   // no part, or one without keys
                continue;
            const float w = exp_of(ml[c].x - m, ml[c].y, lr[c], o[c]);
            Z = fmaf(ml[c].y, w, Z);
            if (kShared)
                Zr = fmaf(lr[c], w, Zr);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                acc[k].x = fmaf(w, o[c][k].x, acc[k].x);
                acc[k].y = fmaf(w, o[c][k].y, acc[k].y);
                acc[k].z = fmaf(w, o[c][k].z, acc[k].z);
                acc[k].w = fmaf(w, o[c][k].w, acc[k].w);
            }
        }
        M = m;
    }
    if (join.y == 0)
        return;
    if (kSplit > 1) {   // the warps' sums, in the order of their runs, by warp k to the dims 128 k ..
        __shared__ float4 mz[kSplit];
        __shared__ float4 sums[kSplit][kLatent / 4];
        if (lane == 0)
            mz[warp] = make_float4(M, Z, Zr, 0.f);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            sums[warp][32 * k + lane] = acc[k];
        __syncthreads();
        if (warp >= 4)
            return;
        float m = -INFINITY;
        for (int i = 0; i < kSplit; ++i)
            m = fmaxf(m, mz[i].x);
        M = m;
        Z = Zr = 0.f;
        acc[0] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = 0; i < kSplit; ++i) {
            if (mz[i].x == -INFINITY)   // (a run without keys)
                continue;
            float4 z = mz[i], o[1] = {sums[i][32 * warp + lane]};
            const float w = z.x == m ? 1.f : exp_of(z.x - m, z.y, z.z, o);
            Z = fmaf(z.y, w, Z);
            Zr = fmaf(z.z, w, Zr);
            acc[0].x = fmaf(w, o[0].x, acc[0].x);
            acc[0].y = fmaf(w, o[0].y, acc[0].y);
            acc[0].z = fmaf(w, o[0].z, acc[0].z);
            acc[0].w = fmaf(w, o[0].w, acc[0].w);
        }
    }
    if (!kShared)
        Zr = Z;
    const float f = Zr > 0.f || Zr != Zr ? 1.f / Zr : 0.f;   // (no key and no sink: zeros)
    const int64_t row = (int64_t)t * p.num_heads + h0 + h;
#pragma unroll
    for (int k = 0; k < (kSplit == 1 ? 4 : 1); ++k)
        *reinterpret_cast<uint2 *>(p.out + row * kLatent + 128 * (kSplit == 1 ? k : warp) + 4 * lane) =
            make_uint2(pack_bf16x2(acc[k].x * f, acc[k].y * f), pack_bf16x2(acc[k].z * f, acc[k].w * f));
    if (lane == 0 && (kSplit == 1 || warp == 0) && p.lse != nullptr)
        p.lse[row] = M == -INFINITY ? -INFINITY : M + logf(Z);
}

}  // namespace

int decode_fp4_block_keys() { return kBK; }
int decode_fp4_own_list_width() { return kListLoads * kListThreads; }
size_t decode_fp4_part_bytes() { return sizeof(float) * (size_t)kPartFloats; }

cudaError_t launch_decode_fp4(const Decode4Params &p, cudaStream_t stream)
{
    if (p.num_tokens <= 0)
        return cudaSuccess;
    if (p.groups != (p.num_heads + kNH - 1) / kNH || p.grid < 1)
        return cudaErrorInvalidValue;
    const bool shared = p.ctas_per_unit > 0;
    const auto kernel = shared ? decode_fp4_kernel<true> : decode_fp4_kernel<false>;
    const cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kernel), kSmemBytes, shared ? kAttrFp4Shared : kAttrFp4);
    if (e != cudaSuccess)
        return e;
    const cudaError_t r = launch_dependent(kernel, dim3((unsigned)p.grid), kThreads, kSmemBytes, stream, p);
    if (r != cudaSuccess || !p.split)
        return r;
    const unsigned units = (unsigned)p.num_tokens * (unsigned)p.groups, heads = (unsigned)std::min(p.num_heads, kNH);
    if (p.ctas_per_unit >= kJoinMany)
        return launch_dependent(join_parts_kernel<2, kJoinSplit, true>, dim3(units, heads), 32 * kJoinSplit, 0, stream, p);
    return launch_dependent(shared ? join_parts_kernel<4, 1, true> : join_parts_kernel<2, 1, false>, dim3(units, heads / kJoinHeads),
                            32 * kJoinHeads, 0, stream, p);
}

}  // namespace dsv4
