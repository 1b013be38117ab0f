// lists_fp4.cu -- the cache slots that each token of a 4-bit decode attends to.
//
// The combine of dsv4_combine_topk_swa_indices (kept top-k entries in input order, then the window
// ascending; entries that are not causal, lie in the window or repeat an earlier one are dropped), with
// every kept position taken through the block table to its cache slot:
//   slots[t][0 .. L) = block_table[row][p / page] * page + p % page  (-1 for a page out of range, which is
//   flagged),  lens[t] = L.   Entries from L on are not written.
//
// One CTA per token.  First occurrences come from a shared-memory hash set of 64-bit slots, (position << 32) |
// smallest top-k index, at most half full: the first writer of a position claims its slot with one CAS, a
// repeat lowers the index; each thread remembers the slots of its first entries.  Ballots over up to four
// passes of the row give the output order.  The steps are dependent latencies (row, set, ballots, table, store);
// a row's entries sit one per thread and pass, so every step is one round for rows of up to 2048 entries.
#include <climits>

#include "fp4.h"

namespace dsv4 {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kPassLoads = 4;
constexpr unsigned long long kEmpty = ~0ull;

__device__ __forceinline__ unsigned hash_pos(int v, int bits) { return ((unsigned)v * 0x9E3779B1u) >> (32 - bits); }

__device__ __forceinline__ unsigned insert(unsigned long long *tab, int bits, int v, int i)
{
    const unsigned long long want = ((unsigned long long)(unsigned)v << 32) | (unsigned)i;
    unsigned h = hash_pos(v, bits);
    while (true) {   // (the set is at most half full)
        const unsigned long long prev = atomicCAS(&tab[h], kEmpty, want);
        if (prev == kEmpty)
            return h;
        if ((unsigned)(prev >> 32) == (unsigned)v) {
            atomicMin(&tab[h], want);
            return h;
        }
        h = (h + 1u) & ((1u << bits) - 1u);
    }
}

__global__ void __launch_bounds__(kThreads) lists_fp4_kernel(const Lists4Params p)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // (the decode waits for this grid itself)
    extern __shared__ unsigned long long tab[];
    __shared__ int wsum[kPassLoads][kWarps];
    const int t = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid < p.groups)
        p.joins[tid * gridDim.x + t] = make_int2(0, 0);
    const int seq_len = p.seq_lens[t];
    const int row = p.req_idx != nullptr ? p.req_idx[t] : t;
    int n = p.topk_width;
    if (p.topk_lens != nullptr) {
        n = p.topk_lens[t];
        n = n < 0 ? 0 : (n > p.topk_width ? p.topk_width : n);
    }
    const int32_t *trow = p.topk + (int64_t)t * p.topk_stride;
    const int npass = (n + kThreads - 1) / kThreads;
    int tv[kPassLoads];
#pragma unroll
    for (int u = 0; u < kPassLoads; ++u)
        tv[u] = u * kThreads + tid < n ? __ldg(trow + u * kThreads + tid) : -1;
    // the set of this row's size
    int bits = 6;
    while ((1 << bits) < 2 * n)
        ++bits;
    const int table = 1 << bits;
    for (int i = tid; i < table; i += kThreads)
        tab[i] = kEmpty;
    const bool row_ok = row >= 0 && row < p.num_reqs;
    const int32_t *bt_row = p.block_table + (int64_t)(row_ok ? row : 0) * p.bt_stride;
    // window [win_lo, pos]; the top-k survivors are the first occurrences of positions in [0, win_lo)
    const int pos = seq_len - 1;   // seq_len <= 0: nothing is visible
    const long long lo = (long long)pos - p.window + 1;
    const int win_lo = lo < 0 ? 0 : (int)lo;
    const int swa = seq_len > 0 ? pos - win_lo + 1 : 0;
    int32_t *out = p.slots + (int64_t)t * p.list_w;
    auto slot_of = [&](int v) {
        const int blk = v / p.page;
        const int phys = row_ok && blk < p.max_blocks ? __ldg(bt_row + blk) : -1;
        if (phys < 0 || phys >= p.num_blocks) {
            atomicOr(p.status, kStatusBadIndex);
            return -1;
        }
        return phys * p.page + (v - blk * p.page);
    };
    __syncthreads();
    unsigned hs[kPassLoads];
#pragma unroll
    for (int u = 0; u < kPassLoads; ++u)
        hs[u] = tv[u] >= 0 && tv[u] < win_lo ? insert(tab, bits, tv[u], u * kThreads + tid) : 0u;
#pragma unroll 1
    for (int ps = kPassLoads; ps < npass; ++ps) {
        const int i = ps * kThreads + tid;
        const int v = i < n ? __ldg(trow + i) : -1;
        if (v >= 0 && v < win_lo)
            insert(tab, bits, v, i);
    }
    // the entries' slots do not depend on which of them are kept
    int sv[kPassLoads];
#pragma unroll
    for (int u = 0; u < kPassLoads; ++u)
        sv[u] = tv[u] >= 0 && tv[u] < win_lo ? slot_of(tv[u]) : -1;
    __syncthreads();
    int total = 0;
#pragma unroll 1
    for (int pg = 0; pg < npass; pg += kPassLoads) {
        unsigned bal[kPassLoads];
        int vg[kPassLoads];
#pragma unroll
        for (int u = 0; u < kPassLoads; ++u) {
            const int i = (pg + u) * kThreads + tid;
            const int v = pg == 0 ? tv[u] : (i < n ? __ldg(trow + i) : -1);
            vg[u] = v;
            bool keep = false;
            if (v >= 0 && v < win_lo) {
                unsigned h = hs[u];
                if (pg != 0) {
                    h = hash_pos(v, bits);
                    while ((unsigned)(tab[h] >> 32) != (unsigned)v)
                        h = (h + 1u) & (unsigned)(table - 1);
                }
                keep = (unsigned)tab[h] == (unsigned)i;
            }
            bal[u] = __ballot_sync(0xffffffffu, keep);
            if (lane == 0)
                wsum[u][warp] = __popc(bal[u]);
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kPassLoads; ++u) {
            const int x = lane < kWarps ? wsum[u][lane] : 0;
            const int before = __reduce_add_sync(0xffffffffu, lane < warp ? x : 0);
            const int rank = total + before + __popc(bal[u] & ((1u << lane) - 1u));
            total += __reduce_add_sync(0xffffffffu, x);
            if ((bal[u] >> lane) & 1u)
                out[rank] = pg == 0 ? sv[u] : slot_of(vg[u]);
        }
        __syncthreads();   // wsum is rewritten by the next group of passes
    }
    for (int k = tid; k < swa; k += kThreads)
        out[total + k] = slot_of(win_lo + k);
    if (tid == 0)
        p.lens[t] = total + swa;
}

}  // namespace

cudaError_t launch_lists_fp4(const Lists4Params &p, cudaStream_t stream)
{
    if (p.num_tokens <= 0)
        return cudaSuccess;
    int bits = 6;
    while ((1 << bits) < 2 * p.topk_width)
        ++bits;
    const int bytes = 8 << bits;
    const cudaError_t e = set_smem_once(reinterpret_cast<const void *>(lists_fp4_kernel), bytes, kAttrFp4Lists);
    if (e != cudaSuccess)
        return e;
    lists_fp4_kernel<<<p.num_tokens, kThreads, bytes, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace dsv4
