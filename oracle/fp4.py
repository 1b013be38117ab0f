"""fp64 CPU oracle of the 4-bit cache and of the page operators (numpy; shares no code with the CUDA library).

TEST INFRASTRUCTURE ONLY, as the rest of this package.  The attention and the index combine are those of oracle.c.
"""
from __future__ import annotations

import numpy as np

import oracle

ENTRY_BYTES, ROPE_OFFSET, SCALE_OFFSET, SCALE_BLOCK = 400, 256, 384, 32
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def bf16_to_f64(bits):
    return (np.asarray(bits, dtype=np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def f64_to_bf16(x):
    """Nearest BF16 bits (ties to even) of finite fp64 values, in one rounding."""
    x = np.asarray(x, dtype=np.float64)
    m, k = np.frexp(np.abs(x))
    step = np.ldexp(1.0, np.maximum(k - 8, -133))
    y = np.copysign(np.rint(np.abs(x) / step) * step, x)
    with np.errstate(over="ignore"):
        return (y.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)


def ue8m0_to_f64(b):
    b = np.asarray(b)
    return np.where(b == 255, np.nan, np.ldexp(1.0, b.astype(np.int64) - 127))


def e2m1_encode(y):
    """E2M1 codes: nearest magnitude, ties to the even code, past 6 -> 6, NaN -> 7."""
    y = np.asarray(y, dtype=np.float64)
    a = np.where(np.isnan(y), np.inf, np.abs(y))
    d = np.abs(np.minimum(a, 1e300)[..., None] - E2M1)
    code = np.where(d[..., 0::2].min(-1) <= d[..., 1::2].min(-1), 2 * d[..., 0::2].argmin(-1), 2 * d[..., 1::2].argmin(-1) + 1)
    code = np.where(a >= 6.0, 7, code)
    return (code | np.where(np.signbit(y) & ~np.isnan(y), 8, 0)).astype(np.uint8)


def exponent(amax):
    """Smallest e in [-127, 125] with 6 * 2^e >= amax (125 past that range); 0 for amax 0."""
    amax = np.asarray(amax, dtype=np.float64)
    es = np.arange(-127, 126)
    ok = 6.0 * np.ldexp(1.0, es) >= amax[..., None]
    e = np.where(ok.any(-1), es[ok.argmax(-1)], 125)
    return np.where(amax == 0, 0, e)


def quantize(latent):
    """fp64 [n, 512] -> (codes uint8 [n, 256], scale bytes uint8 [n, 16])."""
    x = np.asarray(latent, dtype=np.float64).reshape(len(latent), 16, SCALE_BLOCK)
    e = exponent(np.nan_to_num(np.abs(x), nan=0.0, posinf=np.inf).max(-1))
    with np.errstate(invalid="ignore"):
        c = e2m1_encode(x * np.ldexp(1.0, -e)[..., None]).reshape(len(latent), 512)
    return c[:, 0::2] | (c[:, 1::2] << 4), (e + 127).astype(np.uint8)


def pack(latent, rope_bits):
    codes, scales = quantize(latent)
    rope = np.ascontiguousarray(rope_bits).astype("<u2").view(np.uint8).reshape(len(codes), 128)
    return np.concatenate([codes, rope, scales], axis=1)


def dequant(entries):
    """uint8 [n, 400] -> fp64 keys [n, 576]."""
    e = np.ascontiguousarray(entries).reshape(-1, ENTRY_BYTES)
    code = np.stack([e[:, :256] & 15, e[:, :256] >> 4], -1).reshape(-1, 512)
    v = np.where(code & 8, -1.0, 1.0) * E2M1[code & 7]
    with np.errstate(invalid="ignore"):
        v = v * np.repeat(ue8m0_to_f64(e[:, SCALE_OFFSET:]), SCALE_BLOCK, axis=1)
    return np.concatenate([v, bf16_to_f64(np.ascontiguousarray(e[:, ROPE_OFFSET:SCALE_OFFSET]).view("<u2"))], axis=1)


def rotate(x, c, s):
    out = np.empty_like(x)
    out[..., 0::2] = x[..., 0::2] * c - x[..., 1::2] * s
    out[..., 1::2] = x[..., 0::2] * s + x[..., 1::2] * c
    return out


def insert(q_bits, kv_bits, positions, slots, cos_sin, cache, q_w=None, kv_w=None, norm_dims=512, eps=1e-6):
    """-> (q fp64 [T, H, 576], k fp64 before quantisation [T, 576], cache uint8 with the entries, bad count)."""
    q, kv = bf16_to_f64(q_bits), bf16_to_f64(kv_bits)
    cs = np.asarray(cos_sin, dtype=np.float64)
    good = (positions >= 0) & (positions < len(cs))
    at = np.where(good, positions, 0)
    c = np.where(good[:, None], cs[at, :32], 1.0)
    s = np.where(good[:, None], cs[at, 32:], 0.0)
    q = q / np.sqrt((q ** 2).mean(-1, keepdims=True) + eps) * (1.0 if q_w is None else np.asarray(q_w, np.float64))
    q[..., 512:] = rotate(q[..., 512:], c[:, None], s[:, None])
    k, n = kv.copy(), norm_dims
    if n:
        with np.errstate(invalid="ignore", divide="ignore"):
            k[:, :n] = k[:, :n] / np.sqrt((k[:, :n] ** 2).mean(-1, keepdims=True) + eps)
        if kv_w is not None:
            k[:, :n] *= np.asarray(kv_w, np.float64)
    k[:, 512:] = rotate(k[:, 512:], c, s)
    out = np.array(cache, copy=True)
    entries = pack(k[:, :512], f64_to_bf16(k[:, 512:]))
    bad = 0
    for t in range(len(kv)):
        bad += int(not good[t]) + int(slots[t] >= len(out))
        if good[t] and 0 <= slots[t] < len(out):
            out[slots[t]] = entries[t]
    return q, k, out, bad


def decode(w, tokens=None):
    """Decode of a workload whose cache holds 4-bit entries -> (out, lse, sum of weights times |v|, bound of the error
    of a logit's fp32 sum in units of 2^-24, bad count) for the given tokens."""
    T, H, _ = w.q.shape
    tokens = range(T) if tokens is None else tokens
    lists, lens = oracle.combine(w.topk_idx, w.topk_lens, w.seq_lens, w.window, w.topk_idx.shape[1] + w.window)
    n = len(tokens)
    out, mag = np.zeros((n, H, 512)), np.zeros((n, H, 512))
    lse, dot = np.full((n, H), -np.inf), np.zeros((n, H))
    bad = 0
    for i, t in enumerate(tokens):
        row = t if w.req_idx is None else int(w.req_idx[t])
        p = lists[t, :lens[t]].astype(np.int64)
        blk = p // w.page
        key = np.zeros((0, 576))
        if 0 <= row < len(w.block_table):
            ok = blk < w.block_table.shape[1]
            phys = np.where(ok, w.block_table[row, np.minimum(blk, w.block_table.shape[1] - 1)], -1)
            ok &= (phys >= 0) & (phys < len(w.kv_cache))
            key = dequant(w.kv_cache[phys[ok], (p % w.page)[ok]])
            bad += int((~ok).sum())
        else:
            bad += len(p)
        q = bf16_to_f64(w.q[t])
        s = q @ key.T * w.softmax_scale
        if len(key):
            dot[i] = (np.abs(q) @ np.abs(key).T).max(1) * w.softmax_scale
        sk = np.full((H, 1), -np.inf) if w.sink is None else np.asarray(w.sink, np.float64)[:, None]
        every = np.concatenate([s, sk], 1)
        m = every.max(1)
        some = m > -np.inf
        with np.errstate(invalid="ignore", divide="ignore"):
            lse[i] = np.where(some, m + np.log(np.exp(every - m[:, None]).sum(1)), -np.inf)
            wt = np.where(some[:, None], np.exp(s - lse[i][:, None]), 0.0)
        out[i], mag[i] = wt @ key[:, :512], wt @ np.abs(key[:, :512])
    return out, lse, mag, dot, bad


# ---- page operators, one row and one page at a time

def pages(length, page, width):
    return min(width, -(-max(int(length), 0) // page))


def fork(cache, table, lens, refs, parent, share):
    """-> (cache, table, lens, refs, bad) after dsv4_cache_fork_rows; cache [layers, pages, page, bytes]."""
    cache, B, page, M = np.array(cache), cache.shape[1], cache.shape[2], table.shape[1]
    src = np.array(cache)
    free = [b for b in range(B) if refs[b] == 0]
    tout, lout, rout = np.full((len(parent), M), -1, np.int32), np.zeros(len(parent), np.int32), np.array(refs)
    bad, seen, kids, used = 0, set(), {}, 0
    kept = set()
    for r, par in enumerate(parent):
        if par < 0 or par >= len(lens):
            bad += par >= len(lens)
            continue
        L = min(max(int(lens[par]), 0), M * page)
        bad += lens[par] > M * page
        first = par not in seen
        seen.add(par)
        cells, take = [], 0
        for j in range(pages(L, page, M)):
            v = int(table[par, j])
            if not 0 <= v < B:
                bad += 1
                cells.append((j, -1, "bad"))
            elif share and (j + 1) * page <= L:
                cells.append((j, v, "shared"))
            elif first and refs[v] == 1:
                cells.append((j, v, "kept"))
            else:
                cells.append((j, v, "take"))
                take += 1
        at, used = used, used + take
        if take and at + take > len(free):
            bad += 1
            continue
        lout[r] = L
        kids[par] = kids.get(par, 0) + 1
        for j, v, how in cells:
            if how == "take":
                new = free[at]
                at += 1
                n = min(page, L - j * page)
                cache[:, new, :n] = src[:, v, :n]
                tout[r, j], rout[new] = new, 1
            else:
                tout[r, j] = v
                if how == "kept":
                    kept.add((par, j))
    for i in range(len(lens)):                # every row of the table is read, for the references that it gives up or keeps
        L = min(max(int(lens[i]), 0), M * page)
        bad += lens[i] > M * page
        for j in range(pages(L, page, M)):
            v = int(table[i, j])
            bad += not 0 <= v < B
            if 0 <= v < B:
                rout[v] += kids.get(i, 0) - 1 if share and (j + 1) * page <= L else 0 if (i, j) in kept else -1
    return cache, tout, lout, rout, bad


def compact(cache, table, lens, refs):
    """-> (cache, table, refs, page map, live pages, bad) after dsv4_cache_compact."""
    cache, B, page, M = np.array(cache), cache.shape[1], cache.shape[2], table.shape[1]
    live = [b for b in range(B) if refs[b] > 0]
    L = len(live)
    to, rout = np.full(B, -1, np.int32), np.zeros(B, np.int32)
    holes = iter(b for b in range(L) if refs[b] <= 0)
    for b in live:
        to[b] = b if b < L else next(holes)
        rout[to[b]] = refs[b]
        if to[b] != b:
            cache[:, to[b]] = cache[:, b]
    tout, bad = np.full(table.shape, -1, np.int32), 0
    for r in range(len(lens)):
        bad += lens[r] > M * page
        for j in range(pages(lens[r], page, M)):
            v = int(table[r, j])
            tout[r, j] = to[v] if 0 <= v < B else -1
            bad += tout[r, j] < 0
    return cache, tout, rout, to, L, bad


def copy_pages(dst, src, src_pages, dst_pages, one_pool):
    """-> (dst cache, bad) after dsv4_cache_copy_pages."""
    out, bad = np.array(dst), 0
    good = [(i, s, d) for i, (s, d) in enumerate(zip(src_pages, dst_pages)) if 0 <= s < src.shape[1] and 0 <= d < dst.shape[1]]
    bad += len(src_pages) - len(good)
    last = {d: i for i, s, d in good}
    for i, s, d in good:
        if last[d] != i:
            continue
        if one_pool and s in last:
            bad += 1
            continue
        out[:, d] = src[:, s]
    return out, bad
