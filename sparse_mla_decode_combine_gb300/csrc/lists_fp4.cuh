// lists_fp4.cuh -- the cache slots that a token of a 4-bit decode attends to, built by the threads of one CTA.
//
// The combine of dsv4_combine_topk_swa_indices (kept top-k entries in input order, then the window
// ascending; entries that are not causal, lie in the window or repeat an earlier one are dropped), with
// every kept position taken through the block table to its cache slot:
//   slots[t][0 .. L) = block_table[row][p / page] * page + p % page  (-1 for a page out of range, which is
//   flagged).   Entries from L on are not written.
//
// The steps are dependent latencies (row, set, block table, store), so each is one round for rows of up to kLoads entries
// to a thread, and loads that do not depend on one another are issued together.
// Repeats are looked for in a bitmap of the positions (one 32-bit shared-memory OR an entry).  Only a row that has one,
// or positions past the bitmap, goes through a hash set of 64-bit slots, (position << 32) | smallest top-k index, at
// most half full, which says which of the repeats comes first: its 64-bit compare-and-swaps alone took 7 us for 2048
// entries.  Ballots over up to kLoads passes of the row give the output order.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "fp4.h"

namespace dsv4 {
namespace lists {

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

// Token t's list, by kThreads threads (tid: this one's number; whole warps); returns its length.  tab: p.smem_bytes of
// shared memory, wsum: kLoads * kThreads / 32 ints of it.  sync() is a barrier of these threads, sync.any(v) one that
// tells them whether any has v.  range(length) says from which entry to which the window's part of the list is wanted.
// kPositions: p.positions receives the entries' positions beside their slots (-1 as well for a page out of range).
template <int kThreads, int kLoads, bool kPositions = false, typename Sync, typename Range>
__device__ __forceinline__ int build(const Lists4Params &p, int t, int tid, unsigned long long *tab, int *wsum, const Sync &sync,
                                     const Range &range)
{
    constexpr int kWarps = kThreads / 32;
    const int lane = tid & 31, warp = tid >> 5;
    const int32_t *trow = p.topk + (int64_t)t * p.topk_stride;
    int tv[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; ++u)
        tv[u] = u * kThreads + tid < p.topk_width ? __ldca(trow + u * kThreads + tid) : -1;
    const int seq_len = p.seq_lens[t];
    const int row = p.req_idx != nullptr ? p.req_idx[t] : t;
    int n = p.topk_width;
    if (p.topk_lens != nullptr) {
        n = p.topk_lens[t];
        n = n < 0 ? 0 : (n > p.topk_width ? p.topk_width : n);
    }
    const int npass = (n + kThreads - 1) / kThreads;
    const bool row_ok = row >= 0 && row < p.num_reqs;
    const int32_t *bt_row = p.block_table + (int64_t)(row_ok ? row : 0) * p.bt_stride;
    // window [win_lo, pos]; the top-k survivors are the first occurrences of positions in [0, win_lo)
    const int pos = max(seq_len, 0) - 1;   // seq_len <= 0: nothing is visible
    const long long lo = (long long)pos - p.window + 1;
    const int win_lo = lo < 0 ? 0 : (int)lo;
    const int swa = seq_len > 0 ? pos - win_lo + 1 : 0;
    int32_t *out = p.slots + (int64_t)t * p.list_w;
    int32_t *out_pos = kPositions ? p.positions + (int64_t)t * p.list_w : nullptr;
    auto page_at = [&](int blk) { return row_ok && blk < p.max_blocks ? __ldca(bt_row + blk) : -1; };   // (-1: outside the table)
    auto slot_in = [&](int phys, int at) {
        if (phys < 0 || phys >= p.num_blocks) {
            atomicOr(p.status, kStatusBadIndex);
            return -1;
        }
        return phys * p.page + at;
    };
    auto slot_of = [&](int v) {
        const int blk = v / p.page;
        return slot_in(page_at(blk), v - blk * p.page);
    };
#pragma unroll
    for (int u = 0; u < kLoads; ++u)   // entries that are not selectable: -1
        tv[u] = u * kThreads + tid < n && tv[u] >= 0 && tv[u] < win_lo ? tv[u] : -1;

    // ---- is any position listed twice?
    unsigned *seen = reinterpret_cast<unsigned *>(tab);
    bool hashed = win_lo > p.smem_bytes * 8;
    if (!hashed) {
        for (int i = tid; i < (win_lo + 31) / 32; i += kThreads)
            seen[i] = 0u;
        sync();
        bool twice = false;
#pragma unroll
        for (int u = 0; u < kLoads && u * kThreads < n; ++u)
            if (tv[u] >= 0)
                twice |= (atomicOr(&seen[tv[u] >> 5], 1u << (tv[u] & 31)) >> (tv[u] & 31)) & 1u;
#pragma unroll 1
        for (int i = kLoads * kThreads + tid; i < n; i += kThreads) {
            const int v = __ldca(trow + i);
            if (v >= 0 && v < win_lo)
                twice |= (atomicOr(&seen[v >> 5], 1u << (v & 31)) >> (v & 31)) & 1u;
        }
        hashed = sync.any(twice);
    }
    // the entries' slots do not depend on which of them are kept
    int sv[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads && u * kThreads < n; ++u)
        sv[u] = tv[u] >= 0 ? slot_of(tv[u]) : -1;
    int bits = 6;
    while ((1 << bits) < 2 * n)
        ++bits;
    unsigned hs[kLoads];
    if (hashed) {
        for (int i = tid; i < 1 << bits; i += kThreads)
            tab[i] = kEmpty;
        sync();
#pragma unroll
        for (int u = 0; u < kLoads && u * kThreads < n; ++u)
            hs[u] = tv[u] >= 0 ? insert(tab, bits, tv[u], u * kThreads + tid) : 0u;
#pragma unroll 1
        for (int i = kLoads * kThreads + tid; i < n; i += kThreads) {
            const int v = __ldca(trow + i);
            if (v >= 0 && v < win_lo)
                insert(tab, bits, v, i);
        }
        sync();
    }
    int total = 0;
#pragma unroll 1
    for (int pg = 0; pg < npass; pg += kLoads) {
        unsigned bal[kLoads];
        int vg[kLoads];
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            if (pg + u >= npass)
                break;
            const int i = (pg + u) * kThreads + tid;
            int v = pg == 0 ? tv[u] : (i < n ? __ldca(trow + i) : -1);
            v = v < win_lo ? v : -1;
            vg[u] = v;
            bool keep = v >= 0;
            if (keep && hashed) {
                unsigned h = hs[u];
                if (pg != 0) {
                    h = hash_pos(v, bits);
                    while ((unsigned)(tab[h] >> 32) != (unsigned)v)
                        h = (h + 1u) & ((1u << bits) - 1u);
                }
                keep = (unsigned)tab[h] == (unsigned)i;
            }
            bal[u] = __ballot_sync(0xffffffffu, keep);
            if (lane == 0)
                wsum[kWarps * u + warp] = __popc(bal[u]);
        }
        sync();
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            if (pg + u >= npass)
                break;
            const int x = lane < kWarps ? wsum[kWarps * u + lane] : 0;
            const int before = __reduce_add_sync(0xffffffffu, lane < warp ? x : 0);
            const int rank = total + before + __popc(bal[u] & ((1u << lane) - 1u));
            total += __reduce_add_sync(0xffffffffu, x);
            if ((bal[u] >> lane) & 1u) {
                const int slot = pg == 0 ? sv[u] : slot_of(vg[u]);
                out[rank] = slot;
                if (kPositions)
                    out_pos[rank] = slot >= 0 ? vg[u] : -1;
            }
        }
        sync();   // wsum is rewritten by the next group of passes
    }
    const int len = total + swa;
    const int2 part = range(len);
    const int i1 = min(part.y, len);
    int i = max(part.x, total) + tid;
    auto write = [&](int i, int slot) {
        out[i] = slot;
        if (kPositions)
            out_pos[i] = slot >= 0 ? win_lo + (i - total) : -1;
    };
    for (; i + 3 * kThreads < i1; i += 4 * kThreads) {   // the window, four loads in flight
        int phys[4], at[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int v = win_lo + (i - total) + u * kThreads, blk = v / p.page;
            phys[u] = page_at(blk);
            at[u] = v - blk * p.page;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            write(i + u * kThreads, slot_in(phys[u], at[u]));
    }
#pragma unroll 1
    for (; i < i1; i += kThreads)
        write(i, slot_of(win_lo + (i - total)));
    return len;
}

}  // namespace lists
}  // namespace dsv4
