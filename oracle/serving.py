"""fp64 CPU oracle of the operators between two decode steps (numpy, one request, key or row at a time; shares no code with
the CUDA library).

TEST INFRASTRUCTURE ONLY, as the rest of this package.
"""
from __future__ import annotations

import numpy as np

import oracle
from oracle import fp4


def _clean(x):
    x = np.asarray(x, dtype=np.float64)
    return np.where(x > 0, x, 0.0)          # negative values and NaN count as 0


def largest(row):
    """Index of the largest value (the lowest of equal ones, NaN below every number); -1 for a row of NaN."""
    at = -1
    for i, x in enumerate(np.asarray(row, dtype=np.float64)):
        if not np.isnan(x) and (at < 0 or x > row[at]):
            at = i
    return at


def drawn(w, u):
    """-> (token, bounds): the lowest i with w_0 + .. + w_i > u sum(w), and every token whose border lies so near that
    sums good to 2^-44 of the whole could decide for it."""
    total = np.cumsum(np.asarray(w, dtype=np.longdouble))
    want, eps = np.longdouble(u) * total[-1], total[-1] * np.longdouble(2.0) ** -44
    token = int(np.searchsorted(total, want, side="right"))
    before = total - w
    near = np.flatnonzero((w > 0) & (total > want - eps) & (before <= want + eps))
    if token >= len(w):                     # a number of 1 or more: the last one with weight
        token = int(np.flatnonzero(w > 0)[-1])
    return token, set(near.tolist()) | {token}


def verify(target, draft, tokens, start, uniform, greedy=None, seq=None, width=None):
    """-> (tokens, accepted, seq, the tokens that may stand at place a of each request, bad) after dsv4_verify_drafts."""
    V, R = target.shape[1], len(start) - 1
    width = max(1, max(np.diff(start), default=1)) if width is None else width
    out, acc, bad = np.full((R, width), -1, np.int32), np.zeros(R, np.int32), 0
    seq_out = None if seq is None else np.array(seq)
    may = [set() for _ in range(R)]
    for b in range(R):
        r0, n = int(start[b] - start[0]), int(start[b + 1] - start[b])
        d0, k, a = r0 - b, n - 1, 0
        if n < 1 or r0 < 0 or r0 + n > len(target) or d0 < 0 or d0 + k > len(tokens) or n > width:
            bad += 1
            may[b] = {-1}
            continue
        point = -1
        bad += int(np.sum((np.asarray(tokens[d0:d0 + k]) < 0) | (np.asarray(tokens[d0:d0 + k]) >= V)))
        while a < k:
            d, p = int(tokens[d0 + a]), np.asarray(target[r0 + a], dtype=np.float64)
            if greedy is not None and greedy[b]:
                ok = 0 <= d == largest(p)
            elif 0 <= d < V:
                qd = 1.0 if draft is None else float(_clean(draft[d0 + a][d]))
                ok = float(uniform[r0 + a]) * qd < _clean(p[d])
            else:
                ok = False
            if not ok:
                break
            out[b, a] = d
            a += 1
        p = np.asarray(target[r0 + a], dtype=np.float64)
        if greedy is not None and greedy[b]:
            token = largest(p)
            may[b] = {token}
        else:
            w = _clean(p)
            if a < k:
                if draft is None:
                    point = int(tokens[d0 + a])
                    left = np.where(np.arange(V) == point, 0.0, w)
                else:
                    left = _clean(p - _clean(draft[d0 + a]))
                w = left if left.sum() > 0 else w
            token, may[b] = drawn(w, float(uniform[r0 + k])) if 0 < w.sum() < 2.0 ** 127 else (-1, {-1})
        bad += token < 0
        out[b, a], acc[b] = token, a
        if seq is not None:
            seq_out[b] -= k - a
    return out, acc, seq_out, may, bad


def dequant8(entries):
    """uint8 [n, 656] -> fp64 keys [n, 576]."""
    e = np.ascontiguousarray(entries).reshape(-1, 656)
    c = e[:, :512].astype(np.int64)
    x, f = (c >> 3) & 15, c & 7
    v = np.where(x == 0, f * 2.0 ** -9, (1 + f / 8) * np.ldexp(1.0, x - 7))
    v = np.where((c & 127) == 127, np.nan, np.where(c & 128, -v, v))
    with np.errstate(invalid="ignore"):
        v = v * np.repeat(fp4.ue8m0_to_f64(e[:, 640:644]), 128, axis=1)
    return np.concatenate([v, fp4.bf16_to_f64(np.ascontiguousarray(e[:, 512:640]).view("<u2"))], axis=1)


def key_weights(w, lse, table):
    """`table` (fp64 [rows, width]) after dsv4_sparse_mla_key_weights of a workload -> (table, bound, how many
    tokens were added to a place, bad).  `bound`: the largest sum of magnitudes |q| . |k| of a logit, per place times its weight."""
    T, H, _ = w.q.shape
    out, bound, adds, bad = np.array(table, dtype=np.float64), np.zeros(table.shape), np.zeros(table.shape), 0
    lists, lens = oracle.combine(w.topk_idx, w.topk_lens, np.maximum(w.seq_lens, 0), w.window, max(1, w.topk_idx.shape[1] + w.window))
    dequant = dequant8 if w.kv_cache.shape[2] == 656 else fp4.dequant
    for t in range(T):
        row = t if w.req_idx is None else int(w.req_idx[t])
        p = lists[t, :lens[t]].astype(np.int64)
        if not 0 <= row < len(w.block_table):
            bad += len(p)
            continue
        blk = p // w.page
        ok = blk < w.block_table.shape[1]
        phys = np.where(ok, w.block_table[row, np.minimum(blk, w.block_table.shape[1] - 1)], -1)
        ok &= (phys >= 0) & (phys < len(w.kv_cache))
        bad += int((~ok).sum())
        if not ok.any():
            continue
        key, q = dequant(w.kv_cache[phys[ok], (p % w.page)[ok]]), fp4.bf16_to_f64(w.q[t])
        l = np.where(np.isneginf(lse[t]), np.inf, np.asarray(lse[t], np.float64))
        with np.errstate(invalid="ignore", over="ignore"):
            e = np.exp(q @ key.T * w.softmax_scale - l[:, None])
            dot = np.abs(q) @ np.abs(key).T * w.softmax_scale + np.where(np.isinf(l), 0, np.abs(l))[:, None]
        out[row, p[ok]] += e.sum(0)
        bound[row, p[ok]] += (e * dot).sum(0)
        adds[row, p[ok]] += 1
    return out, bound, adds, bad


def evict(cache, table, lens, refs, weights, budget, limit, first, recent):
    """-> (cache, table, lens, refs, weights, bad) after dsv4_cache_evict; cache [layers, pages, page, bytes]."""
    cache, B, page, M = np.array(cache), cache.shape[1], cache.shape[2], table.shape[1]
    old = np.array(cache)
    free = [b for b in range(B) if refs[b] == 0]
    tout, lout, rout = np.full(table.shape, -1, np.int32), np.array(lens), np.array(refs)
    wout, bad, used = np.zeros_like(weights), 0, 0
    for r in range(len(lens)):
        n = min(max(int(lens[r]), 0), M * page)
        bad += lens[r] > M * page
        have = fp4.pages(n, page, M)
        cells = [int(v) if 0 <= v < B else -1 for v in table[r, :have]]
        bad += cells.count(-1)
        lout[r], tout[r, :have], wout[r, :n] = n, cells, weights[r, :n]
        if n <= limit:
            continue
        between = sorted(range(first, n - recent),
                         key=lambda i: (np.isnan(weights[r, i]), -weights[r, i] if not np.isnan(weights[r, i]) else 0, i))
        keep = sorted(list(range(first)) + between[:budget - first - recent] + list(range(n - recent, n)))
        assert len(keep) == budget
        new, need = [], 0
        for j in range(fp4.pages(budget, page, M)):
            stays = (j + 1) * page <= budget and all(keep[i] == i for i in range(j * page, (j + 1) * page))
            take = cells[j] >= 0 and not stays and refs[cells[j]] != 1
            new.append(None if take else cells[j])
            need += take
        at, used = used, used + need
        if need and at + need > len(free):
            bad += 1
            continue
        for j, v in enumerate(new):
            if v is None:
                new[j] = free[at]
                rout[free[at]] = 1
                rout[cells[j]] -= 1
                at += 1
        for v in cells[len(new):]:
            if v >= 0:
                rout[v] -= 1
        for i, k in enumerate(keep):
            a, b = cells[k // page], new[i // page]
            if a >= 0 and b >= 0:
                cache[:, b, i % page] = old[:, a, k % page]
        lout[r] = budget
        tout[r], wout[r] = -1, 0
        tout[r, :len(new)], wout[r, :budget] = new, weights[r, keep]
    return cache, tout, lout, rout, wout, bad
