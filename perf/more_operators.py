"""What a serving loop does between two decode steps: verify the drafted tokens of each request, credit the cache's keys
with the attention weight that they received, and evict the lightest keys of rows that have grown past their budget.

`own` chooses between the framework's kernels (true) and the plain form in elementary torch operations (false).  The
plain forms compute in 32 bits and round once at the end; the sums that a drawn token is looked up in, and the products
that a draft is accepted by, are taken in 64 bits, since a draw next to a border is decided by them.

Cache entries: 656 bytes (512 E4M3 latent codes, 64 BF16 rope values, 4 UE8M0 scale bytes of 128 values each, padding)
or 400 bytes (512 E2M1 codes, 64 BF16 rope values, 16 UE8M0 scale bytes of 32 values each).
"""
import math

import numpy as np
import torch

own = False

ENTRY4, ENTRY8 = 400, 656
DIM, LATENT, ROPE = 576, 512, 64
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)      # magnitudes of the E2M1 codes 0..7


# --------------------------------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------------------------------
def listed():
    return [
        # one interactive request with three drafts: latency is all there is
        dict(name="verify-one", op="verify", reqs=1, k_lo=3, k_hi=3, vocab=32000, dtype="float32", drafts="probs",
             greedy=0.0, noise=0.7),
        # an ordinary batch: ragged numbers of drafts, an odd vocabulary, a third of the requests greedy
        dict(name="verify-mixed", op="verify", reqs=48, k_lo=0, k_hi=5, vocab=100277, dtype="bfloat16", drafts="probs",
             greedy=0.33, noise=0.7),
        # a large batch whose drafts come without probabilities
        dict(name="verify-points", op="verify", reqs=160, k_lo=2, k_hi=2, vocab=128000, dtype="float32", drafts="points",
             greedy=0.0, noise=0.3),
        # the largest batch: two rows of probabilities to a request that is turned down
        dict(name="verify-large", op="verify", reqs=256, k_lo=1, k_hi=3, vocab=151937, dtype="float32", drafts="probs",
             greedy=0.0, noise=0.9),
        # one small request batch
        dict(name="weights-tiny", op="weights", tokens=2, per_req=1, heads=16, seq_lo=256, seq_hi=256, topk=64,
             ragged=False, window=32, page=64, pad=0, entry=ENTRY8),
        # an ordinary decode batch over the 4-bit cache
        dict(name="weights-mid", op="weights", tokens=32, per_req=1, heads=64, seq_lo=8192, seq_hi=8192, topk=512,
             ragged=False, window=128, page=64, pad=0, entry=ENTRY4),
        # speculative verification: two tokens of a request credit one row
        dict(name="weights-verify", op="weights", tokens=128, per_req=2, heads=128, seq_lo=4096, seq_hi=65536, topk=2048,
             ragged=True, window=128, page=64, pad=0, entry=ENTRY8),
        # a few long histories, attended to as a whole
        dict(name="weights-dense", op="weights", tokens=6, per_req=1, heads=128, seq_lo=20001, seq_hi=40000, topk=0,
             ragged=False, window=40000, page=64, pad=1, entry=ENTRY4),
        # a handful of short rows, in one layer
        dict(name="evict-small", op="evict", groups=4, beams=1, len_lo=300, len_hi=700, budget=256, limit=256, first=4,
             recent=32, page=16, entry=ENTRY4, layers=1, spare=16, unseen=0.3),
        # sampled continuations that share their prompts' pages: shared pages are left to the others
        dict(name="evict-shared", op="evict", groups=8, beams=4, len_lo=1500, len_hi=2500, budget=1001, limit=1200, first=4,
             recent=128, page=64, entry=ENTRY8, layers=4, spare=600, unseen=0.5),
        # one long document cut to a quarter
        dict(name="evict-long", op="evict", groups=1, beams=1, len_lo=131000, len_hi=131000, budget=32768, limit=65536,
             first=16, recent=1024, page=64, entry=ENTRY4, layers=4, spare=16, unseen=0.6),
        # a full batch of long rows in eight layers, some of them still below the limit
        dict(name="evict-large", op="evict", groups=64, beams=1, len_lo=3500, len_hi=12000, budget=4096, limit=4096, first=4,
             recent=512, page=64, entry=ENTRY4, layers=8, spare=16, unseen=0.5),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("verify", "weights", "evict"))
    if op == "verify":
        reqs, k_hi = _log(rng, 1, 250), rng.choice((0, 1, 2, 3, 4, 7))
        most = 100_000_000 // (reqs * (k_hi + 1))
        return dict(op=op, reqs=reqs, k_lo=rng.randint(0, k_hi), k_hi=k_hi, vocab=_log(rng, 900, min(150000, most)),
                    dtype=rng.choice(("float32", "bfloat16")), drafts=rng.choice(("probs", "probs", "points")),
                    greedy=rng.choice((0.0, 0.0, 0.5, 1.0)), noise=rng.choice((0.1, 0.5, 1.0)))
    if op == "weights":
        per_req = rng.choice((1, 1, 2, 3))
        reqs = _log(rng, 1, 126 // per_req)
        seq_hi = min(_log(rng, 48, 131072), 4_000_000 // reqs)
        dense = rng.random() < 0.25 and reqs * per_req * seq_hi <= 250_000
        return dict(op=op, tokens=reqs * per_req, per_req=per_req, heads=rng.choice((16, 32, 64, 128)),
                    seq_lo=max(per_req, seq_hi // rng.choice((1, 4, 16))), seq_hi=seq_hi,
                    topk=0 if dense else _log(rng, 16, 2048), ragged=not dense and rng.random() < 0.5,
                    window=seq_hi if dense else rng.choice((0, 1, 17, 64, 100, 128)), page=rng.choice((16, 32, 64, 256)),
                    pad=rng.choice((0, 0, 1, 3)), entry=rng.choice((ENTRY4, ENTRY8)))
    groups = _log(rng, 1, 40)
    beams = rng.choice((1, 1, 2, 4))
    len_hi = min(_log(rng, 100, 60000), 200_000 // (groups * beams))
    budget = max(8, int(len_hi * rng.uniform(0.1, 0.9)))
    first = rng.choice((0, 1, 4, min(64, budget // 4)))
    page = rng.choice((16, 32, 64))
    return dict(op=op, groups=groups, beams=beams, len_lo=max(1, int(len_hi * rng.uniform(0.1, 0.9))), len_hi=len_hi,
                budget=budget, limit=budget + rng.choice((0, 0, len_hi // 8)), first=first,
                recent=rng.choice((0, 1, budget // 4, budget - first)), page=page,
                entry=rng.choice((ENTRY4, ENTRY4, ENTRY8)), layers=rng.choice((1, 2, 3, 5)),
                spare=groups * beams * (budget // page + 1) if beams > 1 else 4, unseen=rng.uniform(0.0, 0.8))


# --------------------------------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------------------------------
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _prepare_verify(c, seed):
    g, r = _generator(seed), np.random.default_rng(seed)
    R, V, dtype = c["reqs"], c["vocab"], getattr(torch, c["dtype"])
    k = r.integers(c["k_lo"], c["k_hi"], size=R, endpoint=True)
    start = np.concatenate([[0], np.cumsum(k + 1)])
    N, Nd = int(start[-1]), int(k.sum())
    target = torch.empty(N, V, dtype=dtype, device="cuda")
    draft = torch.empty(Nd, V, dtype=dtype, device="cuda") if c["drafts"] == "probs" else None
    tokens = torch.empty(Nd, dtype=torch.int32, device="cuda")
    # a language model's probabilities: few likely tokens and a long tail; the draft model's are near them
    likely = torch.randn(V, generator=g, device="cuda") * 2.0
    at = 0
    for b in range(R):
        rows = int(k[b]) + 1
        z = torch.randn(rows, V, generator=g, device="cuda") * 2.0 + likely
        target[start[b]:start[b] + rows] = torch.softmax(z, 1).to(dtype)
        if rows > 1:
            y = z[:-1] + torch.randn(rows - 1, V, generator=g, device="cuda") * c["noise"]
            if draft is not None:
                draft[at:at + rows - 1] = torch.softmax(y, 1).to(dtype)
                y = y - torch.log(-torch.log(torch.rand(rows - 1, V, generator=g, device="cuda").clamp(1e-9, 1 - 1e-6)))
            tokens[at:at + rows - 1] = y.argmax(1).to(torch.int32)           # a draw from the draft, or its likeliest token
            at += rows - 1
    seq = r.integers(c["k_hi"] + 1, 60000, size=R).astype(np.int32)
    return dict(op="verify", target=target, draft=draft, tokens=tokens, start=_dev(start.astype(np.int32)),
                uniform=torch.rand(N, generator=g, device="cuda"), greedy=_dev((r.random(R) < c["greedy"]).astype(np.uint8)),
                seq=_dev(seq), out=torch.empty(R, c["k_hi"] + 1, dtype=torch.int32, device="cuda"),
                accepted=torch.empty(R, dtype=torch.int32, device="cuda"),
                seq_out=torch.empty(R, dtype=torch.int32, device="cuda"))


def _entries4(x, rope):
    """Real 4-bit entries of random latents: what a cache in use holds."""
    x = x.double().view(-1, 16, 32)
    m, k = torch.frexp(x.abs().amax(-1) / 6.0)              # amax / 6 = m 2^k, 1/2 <= m < 1
    e = torch.where(m > 0.5, k, k - 1)
    y = torch.ldexp(x, -e[..., None])
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device=x.device)
    code = torch.bucketize(y.abs(), mids)
    code = (code | (torch.signbit(y).to(code.dtype) << 3)).view(-1, LATENT).to(torch.uint8)
    return torch.cat([code[:, 0::2] | (code[:, 1::2] << 4), rope, (e + 127).to(torch.uint8)], 1)


def _entries8(x, rope):
    """Real 8-bit entries of random latents."""
    x = x.double().view(-1, 4, 128)
    m, k = torch.frexp(x.abs().amax(-1) / 448.0)
    e = torch.where(m > 0.5, k, k - 1)
    code = torch.ldexp(x, -e[..., None]).float().view(-1, LATENT).to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.cat([code, rope, (e + 127).to(torch.uint8), torch.zeros(len(code), 12, dtype=torch.uint8, device=x.device)], 1)


def _cache(g, slots, entry):
    """A cache whose entries are draws from a pool of quantised rows."""
    n = min(slots, 8192)
    x = torch.randn(n, LATENT, generator=g, device="cuda")
    rope = torch.randn(n, ROPE, generator=g, device="cuda").bfloat16().view(torch.uint8)
    pool = _entries4(x, rope) if entry == ENTRY4 else _entries8(x, rope)
    out = torch.empty(slots, entry, dtype=torch.uint8, device="cuda")
    for lo in range(0, slots, 1 << 20):                     # (in parts, for the index's sake)
        hi = min(slots, lo + (1 << 20))
        out[lo:hi] = pool[torch.randint(0, n, (hi - lo,), generator=g, device="cuda")]
    return out


def _prepare_weights(c, seed):
    g, r = _generator(seed), np.random.default_rng(seed)
    reqs = c["tokens"] // c["per_req"]
    pad, page, K, H = c["pad"], c["page"], c["topk"], c["heads"]
    lens = r.integers(c["seq_lo"], c["seq_hi"], size=reqs, endpoint=True)
    pages = -(-lens // page)
    table = np.full((reqs, -(-c["seq_hi"] // page)), -1, dtype=np.int32)
    perm, at = r.permutation(int(pages.sum())).astype(np.int32), 0
    for i, n in enumerate(pages):
        table[i, :n] = perm[at:at + n]
        at += n
    pos = np.concatenate([np.arange(s - c["per_req"], s) for s in lens])
    T = c["tokens"] + pad                                   # padding tokens see nothing
    seq = _dev(np.concatenate([pos + 1, np.zeros(pad)]).astype(np.int32))
    req = _dev(np.concatenate([np.repeat(np.arange(reqs), c["per_req"]), np.zeros(pad)]).astype(np.int32))
    idx, lens_k = torch.empty(T, 0, dtype=torch.int32, device="cuda"), None
    if K:
        score = torch.rand(T, max(K, c["seq_hi"]), generator=g, device="cuda")
        score.masked_fill_(torch.arange(score.shape[1], device="cuda") >= seq[:, None], -1.0)
        best, idx = score.topk(K, dim=1)                    # distinct positions in random order
        idx = torch.where(best >= 0, idx, -1).to(torch.int32)
        n = (best >= 0).sum(1).to(torch.int32)
        if c["ragged"]:
            lens_k = torch.minimum(n, torch.randint(max(1, K // 8), K + 1, (T,), generator=g, device="cuda",
                                                    dtype=torch.int32))
            idx = torch.where(torch.arange(K, device="cuda") < lens_k[:, None], idx, -1)
    s = dict(op="weights", q=torch.randn(T, H, DIM, generator=g, device="cuda").bfloat16(),
             cache=_cache(g, int(pages.sum()) * page, c["entry"]).view(-1, page, c["entry"]), table=_dev(table), req=req,
             topk=idx.contiguous(), topk_lens=lens_k, seq=seq, window=c["window"], scale=1.0 / math.sqrt(DIM),
             workspace=None)
    s["lse"] = torch.empty(T, H, device="cuda")
    for t in range(T):                                      # what the decode of these tokens returned
        p, ok = _lists({**s, "topk": s["topk"][t:t + 1], "seq": seq[t:t + 1],
                        "topk_lens": None if lens_k is None else lens_k[t:t + 1]})
        z = _logits(s, p, req[t:t + 1], s["q"][t:t + 1]).masked_fill(~ok[:, None], -torch.inf)
        s["lse"][t] = torch.logsumexp(z.double(), -1)[0].float()
    # the weights of the steps before this one: a few keys have most of them
    s["weights"] = torch.randn(reqs, table.shape[1] * page, generator=g, device="cuda").mul_(1.5).exp_().mul_(0.01)
    s["weights"].masked_fill_(torch.arange(table.shape[1] * page, device="cuda") >= _dev(lens)[:, None], 0.0)
    if own:
        import sparse_mla_decode_combine_gb300 as pkg
        s["workspace"] = pkg.workspace_for_key_weights(T, H, K, c["window"])
    return s


def _prepare_evict(c, seed):
    g, r = _generator(seed), np.random.default_rng(seed)
    page, beams = c["page"], c["beams"]
    lens, held = [], []                                     # rows' lengths, and how many pages of each are its group's
    for _ in range(c["groups"]):
        prompt = int(r.integers(c["len_lo"], c["len_hi"], endpoint=True)) if beams == 1 else \
            int(r.integers(max(1, c["len_lo"] // 2), c["len_lo"], endpoint=True))
        for _ in range(beams):
            lens.append(prompt if beams == 1 else int(r.integers(max(prompt, c["len_lo"]), c["len_hi"], endpoint=True)))
            held.append(0 if beams == 1 else prompt // page)
    lens = np.array(lens, dtype=np.int32)
    pages = -(-lens // page)
    most = -(-c["len_hi"] // page)
    blocks = len(lens) * most + c["spare"]
    perm, at = r.permutation(blocks).astype(np.int32), 0
    table = np.full((len(lens), most + 2), -1, dtype=np.int32)               # rows have room to grow
    for i, n in enumerate(pages):
        if i % beams == 0:
            head = perm[at:at + held[i]]
            at += held[i]
        table[i, :held[i]] = head
        table[i, held[i]:n] = perm[at:at + n - held[i]]
        at += n - held[i]
    refs = np.bincount(table[table >= 0], minlength=blocks).astype(np.int32)
    R, width = len(lens), table.shape[1] * page
    # accumulated weights: a few keys have most, and many were never listed
    w = torch.randn(R, width, generator=g, device="cuda").mul_(2.0).exp_()
    w.masked_fill_(torch.rand(R, width, generator=g, device="cuda") < c["unseen"], 0.0)
    w.masked_fill_(torch.arange(width, device="cuda") >= _dev(lens)[:, None], 0.0)
    s = dict(op="evict", weights=w, table=_dev(table), lens=_dev(lens), refs=_dev(refs), budget=c["budget"],
             limit=c["limit"], first=c["first"], recent=c["recent"],
             cache=torch.randint(0, 256, (c["layers"], blocks, page, c["entry"]), dtype=torch.uint8, generator=g,
                                 device="cuda"),
             table_out=torch.empty(table.shape, dtype=torch.int32, device="cuda"),
             lens_out=torch.empty(R, dtype=torch.int32, device="cuda"),
             refs_out=torch.empty(blocks, dtype=torch.int32, device="cuda"), weights_out=torch.empty_like(w),
             workspace=None)
    if own:
        import sparse_mla_decode_combine_gb300 as pkg
        s["workspace"] = pkg.workspace_for_cache_evict(R, table.shape[1], blocks, c["layers"], page, c["entry"], c["budget"])
    return s


def prepare(case, seed):
    return {"verify": _prepare_verify, "weights": _prepare_weights, "evict": _prepare_evict}[case["op"]](case, seed)


# --------------------------------------------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------------------------------------------
def _verify(s):
    p, q, u, start = s["target"], s["draft"], s["uniform"].double(), s["start"].long()
    R, V, dev = start.numel() - 1, p.shape[1], p.device
    k = start[1:] - start[:-1] - 1
    j = torch.arange(s["out"].shape[1], device=dev)
    there = j < k[:, None]                                                   # draft j of request b
    row = torch.where(there, start[:-1, None] + j, 0)
    drow = torch.where(there, start[:-1, None] - torch.arange(R, device=dev)[:, None] + j, 0)
    tok = s["tokens"][drow].long() if s["tokens"].numel() else torch.zeros_like(drow)
    pd = p[row, tok].double()
    qd = torch.ones_like(pd) if q is None else q[drow, tok].double() if q.shape[0] else torch.zeros_like(pd)
    ids = torch.arange(V, device=dev)
    greedy = s["greedy"].bool()
    good = u[row] * qd < pd
    best = None
    if bool(greedy.any()):
        best = torch.where(p == p.amax(1, keepdim=True), ids, V).amin(1)     # ties: the lowest
        good = torch.where(greedy[:, None], best[row] == tok, good)
    a = ((good & there).long().cumprod(1)).sum(1)
    last = start[:-1] + a
    w = p[last].double()                                                     # the row that the next token comes from
    at = a.clamp(max=j.numel() - 1)
    down = (a < k)[:, None]                                                  # turned down: what the draft had is taken off
    of = drow.gather(1, at[:, None])[:, 0]
    if q is None:
        less = torch.where(ids == tok.gather(1, at[:, None]), torch.inf, 0.0)
        w = torch.where(down, (w - less).clamp(min=0), w)
    elif q.shape[0]:
        w = torch.where(down, (w - q[of].double()).clamp(min=0), w)
    total = w.cumsum(1)
    new = (total <= u[start[1:] - 1, None] * total[:, -1:]).sum(1)
    if best is not None:
        new = torch.where(greedy, best[last], new)
    out = torch.where(j < a[:, None], tok, torch.where(j == a[:, None], new[:, None], -1))
    return {"tokens": out.int(), "accepted": a.int(), "seq": s["seq"] - (k - a).int()}


def _dequantised(entries):
    """uint8 [..., 400 or 656] -> float32 keys [..., 576]."""
    if entries.shape[-1] == ENTRY4:
        grid = torch.tensor(GRID + tuple(-v for v in GRID), device=entries.device)
        codes = entries[..., :256]
        latent = torch.stack([grid[(codes & 15).long()], grid[(codes >> 4).long()]], -1).flatten(-2)
        scale, rope = entries[..., 384:], entries[..., 256:384]
    else:
        latent = entries[..., :512].contiguous().view(torch.float8_e4m3fn).float()
        scale, rope = entries[..., 640:644], entries[..., 512:640]
    n = scale.shape[-1]
    latent = (latent.unflatten(-1, (n, LATENT // n)) * torch.exp2(scale.float() - 127.0)[..., None]).flatten(-2)
    return torch.cat([latent, rope.contiguous().view(torch.bfloat16).float()], -1)


def _lists(s):
    """Each token's positions [T, K + W], and which of them are keys."""
    topk, W = s["topk"].long(), s["window"]
    T, K = topk.shape
    dev = topk.device
    pos = s["seq"].long() - 1
    lo = (pos - W + 1).clamp(min=0)
    n = torch.full_like(pos, K) if s["topk_lens"] is None else s["topk_lens"].long().clamp(0, K)
    ok = (torch.arange(K, device=dev) < n[:, None]) & (topk >= 0) & (topk < lo[:, None])
    if K:
        srt, order = torch.where(ok, topk, -1).sort(dim=1, stable=True)      # repeats: the first one stays
        fresh = torch.cat([torch.ones(T, 1, dtype=torch.bool, device=dev), srt[:, 1:] != srt[:, :-1]], 1)
        ok &= torch.zeros_like(ok).scatter(1, order, fresh)
    win = lo[:, None] + torch.arange(W, device=dev)
    ok = torch.cat([ok, win <= pos[:, None]], 1)
    return torch.where(ok, torch.cat([topk, win], 1), 0), ok


def _logits(s, p, req, q):
    page = s["cache"].shape[1]
    block = s["table"][req.long()[:, None], p // page].long().clamp(min=0)
    k = _dequantised(s["cache"][block, p % page])
    return torch.matmul(q.float(), k.transpose(1, 2)) * s["scale"]


def _weights(s):
    p, ok = _lists(s)
    e = torch.exp(_logits(s, p, s["req"], s["q"]) - torch.where(s["lse"] == -torch.inf, torch.inf, s["lse"])[..., None])
    got = e.sum(1)[ok]
    rows = s["req"].long()[:, None].expand_as(p)[ok]
    s["weights"].index_put_((rows, p[ok]), got, accumulate=True)
    return {"weights": s["weights"]}


def _evict(s):
    w, table, refs, n = s["weights"], s["table"], s["refs"], s["lens"].long()
    page, M, dev = s["cache"].shape[2], table.shape[1], table.device
    R, width = w.shape
    budget, first, recent = s["budget"], s["first"], s["recent"]
    cut = n > s["limit"]
    m = torch.where(cut, budget, n)
    i = torch.arange(width, device=dev)
    must = (i < first) | (i >= n[:, None] - recent)
    score = torch.where(must, torch.inf, w).masked_fill(i >= n[:, None], -torch.inf)
    order = score.sort(dim=1, descending=True, stable=True).indices          # the heaviest first, ties by position
    keep = torch.zeros(R, width, dtype=torch.bool, device=dev).scatter(1, order, i < m[:, None])
    src = torch.where(keep, i, width).sort(dim=1).values                     # kept positions in order, then `width`
    live = i < m[:, None]
    src = torch.where(live, src, 0)
    # pages: those whose entries all stay where they are stay, the others are written where the row alone holds them
    j = torch.arange(M, device=dev)
    np_old, np_new = -(-n // page), -(-m // page)
    moved = (live & (src != i)).unflatten(1, (M, page)).any(2) | ((j + 1) * page > m[:, None])
    moved &= (j < np_new[:, None]) & cut[:, None]
    need = moved & (refs[table.clamp(min=0).long()] != 1)
    free = (refs != 0).sort(stable=True).indices                             # the free pages first, lowest first
    new = free[(need.flatten().cumsum(0) - 1).clamp(min=0)].view(need.shape)
    out = torch.where(need, new, torch.where(j < np_new[:, None], table.long(), -1))
    gone = (j < np_old[:, None]) & (need | (j >= np_new[:, None]))
    refs_out = refs.clone()
    refs_out.index_put_((table[gone].long(),), torch.full((1,), -1, dtype=torch.int32, device=dev), accumulate=True)
    refs_out[new[need]] = 1
    go = live & (moved | need).repeat_interleave(page, 1)                    # entries that are written
    r = torch.arange(R, device=dev)[:, None].expand_as(src)[go]
    a, b = src[go], i.expand_as(src)[go]
    flat = s["cache"].view(s["cache"].shape[0], -1, s["cache"].shape[3])
    flat[:, out[r, b // page] * page + b % page] = flat[:, table[r, a // page].long() * page + a % page]
    return {"table": out.int(), "lens": m.int(), "refs": refs_out,
            "weights": torch.where(live, w.gather(1, src), 0.0), "cache": s["cache"]}


def run(state):
    s = state
    if own:
        import sparse_mla_decode_combine_gb300 as pkg
        if s["op"] == "verify":
            pkg.check(pkg.dsv4_verify_drafts(s["target"], s["draft"], s["tokens"], s["start"], s["uniform"], s["out"],
                                             s["accepted"], s["greedy"], s["seq"], s["seq_out"]))
            return {"tokens": s["out"], "accepted": s["accepted"], "seq": s["seq_out"]}
        if s["op"] == "weights":
            pkg.check(pkg.dsv4_sparse_mla_key_weights(s["q"], s["cache"], s["table"], s["req"], s["topk"], s["topk_lens"],
                                                      s["seq"], s["window"], s["lse"], s["scale"], s["weights"],
                                                      s["workspace"]))
            return {"weights": s["weights"]}
        pkg.check(pkg.dsv4_cache_evict(s["cache"], s["table"], s["lens"], s["refs"], s["weights"], s["budget"], s["limit"],
                                       s["first"], s["recent"], s["table_out"], s["lens_out"], s["refs_out"],
                                       s["weights_out"], s["workspace"]))
        return {"table": s["table_out"], "lens": s["lens_out"], "refs": s["refs_out"], "weights": s["weights_out"],
                "cache": s["cache"]}
    return {"verify": _verify, "weights": _weights, "evict": _evict}[s["op"]](s)


# --------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "verify":
        # a request reads the row that its next token comes from, with the draft's row where a draft was turned down; a
        # greedy one the rows up to there.  Half of the drafts of a step are taken as accepted.
        size = 4 if c["dtype"] == "float32" else 2
        k = (c["k_lo"] + c["k_hi"]) / 2
        down = 1 - 0.5 ** k
        rows = (1 - c["greedy"]) * (1 + (down if c["drafts"] == "probs" else 0)) + c["greedy"] * sum(
            0.5 ** i for i in range(int(round(k)) + 1))
        return {"bytes": c["reqs"] * (rows * c["vocab"] * size + 20 * (k + 1)), "flops": c["reqs"] * rows * c["vocab"]}
    if c["op"] == "weights":
        T, H = c["tokens"] + c["pad"], c["heads"]
        seq = (c["seq_lo"] + c["seq_hi"]) / 2
        win = min(c["window"], seq)
        picks = c["topk"] * (9 / 16 if c["ragged"] else 1.0)
        picks = min(picks * max(0.0, 1 - win / seq) if c["topk"] < seq else seq, max(0.0, seq - win))
        keys = c["tokens"] * (picks + win)
        return {"bytes": keys * (c["entry"] + 8) + T * H * (2 * DIM + 4) + 4 * T * c["topk"], "flops": 2 * keys * H * DIM}
    rows, L = c["groups"] * c["beams"], c["layers"]
    lo, hi = c["len_lo"], c["len_hi"]
    cut = 1.0 if lo > c["limit"] else max(0.0, (hi - c["limit"]) / max(1, hi - lo))   # share of rows that are cut
    n = (lo + hi) / 2
    return {"bytes": rows * (cut * 2 * max(0, c["budget"] - c["first"]) * c["entry"] * L + 4 * (2 * n + 3 * n / c["page"])),
            "flops": 0}


# --------------------------------------------------------------------------------------------------------------
# the operators from their definitions, in 64 bits
# --------------------------------------------------------------------------------------------------------------
def _exact_verify(s):
    start, toks, greedy, seq = (s[n].cpu().numpy() for n in ("start", "tokens", "greedy", "seq"))
    u = s["uniform"].double().cpu().numpy()
    R, width = len(start) - 1, s["out"].shape[1]
    out, accepted = np.full((R, width), -1, np.int32), np.zeros(R, np.int32)
    row_of = lambda m, i: m[i].double().cpu().numpy()  # noqa: E731
    for b in range(R):
        k, r0, d0 = int(start[b + 1] - start[b]) - 1, int(start[b]), int(start[b]) - b
        a = 0
        while True:
            p = row_of(s["target"], r0 + a)
            if a == k:
                w = p
                break
            d = int(toks[d0 + a])
            if greedy[b]:
                ok = int(np.flatnonzero(p == p.max())[0]) == d
            else:
                ok = u[r0 + a] * (1.0 if s["draft"] is None else float(s["draft"][d0 + a, d])) < p[d]
            if not ok:
                w = p.copy()
                if s["draft"] is None:
                    w[d] = 0.0
                else:
                    w = np.maximum(p - row_of(s["draft"], d0 + a), 0.0)
                break
            out[b, a] = d
            a += 1
        if greedy[b]:
            out[b, a] = np.flatnonzero(p == p.max())[0]
        else:
            total = np.cumsum(w)
            out[b, a] = np.searchsorted(total, u[r0 + k] * total[-1], side="right")
        accepted[b] = a
    return {"tokens": out, "accepted": accepted, "seq": seq - (start[1:] - start[:-1] - 1 - accepted).astype(np.int32)}


def _exact_key(raw):
    """uint8 numpy [n, 400 or 656] -> float64 keys [n, 576], byte by byte from the formats."""
    key = np.empty((raw.shape[0], DIM))
    if raw.shape[1] == ENTRY4:
        value = np.array([(-1.0 if code & 8 else 1.0) * (0.5 * (code & 1) if (code >> 1) & 3 == 0 else
                          (1 + 0.5 * (code & 1)) * 2.0 ** (((code >> 1) & 3) - 1)) for code in range(16)])
        key[:, 0:LATENT:2], key[:, 1:LATENT:2] = value[raw[:, :256] & 15], value[raw[:, :256] >> 4]
        scales, block, rope = raw[:, 384:], 32, raw[:, 256:384]
    else:
        value = np.array([(-1.0 if code & 128 else 1.0) * ((code & 7) * 2.0 ** -9 if (code >> 3) & 15 == 0 else
                          (1 + (code & 7) / 8) * 2.0 ** (((code >> 3) & 15) - 7)) for code in range(256)])
        value[[127, 255]] = np.nan
        key[:, :LATENT] = value[raw[:, :512]]
        scales, block, rope = raw[:, 640:644], 128, raw[:, 512:640]
    key[:, :LATENT] *= np.repeat(np.ldexp(1.0, scales.astype(np.int64) - 127), block, axis=1)
    key[:, LATENT:] = (rope.copy().view("<u2").astype(np.uint32) << 16).view(np.float32)
    return key


def _exact_weights(s):
    topk, seq, req, table = (s[k].cpu().numpy() for k in ("topk", "seq", "req", "table"))
    lens = None if s["topk_lens"] is None else s["topk_lens"].cpu().numpy()
    total, page, lse = s["weights"].double(), s["cache"].shape[1], s["lse"].double()
    for t in range(len(seq)):
        pos = int(seq[t]) - 1
        lo = max(0, pos - s["window"] + 1)
        picks = topk[t] if lens is None else topk[t, :lens[t]]
        picks = list(dict.fromkeys(int(p) for p in picks if 0 <= p < lo)) + list(range(lo, pos + 1))
        for at in range(0, len(picks), 16384):
            p = np.array(picks[at:at + 16384])
            raw = s["cache"][_dev(table[req[t], p // page].astype(np.int64)), _dev(p % page)].cpu().numpy()
            z = (s["q"][t].double() @ torch.from_numpy(_exact_key(raw)).cuda().T) * s["scale"]
            total[int(req[t])].index_add_(0, _dev(p), torch.exp(z - lse[t][:, None]).sum(0))
    return {"weights": total}


def _exact_evict(s):
    w, lens = s["weights"].double().cpu().numpy(), s["lens"].cpu().numpy()
    new, out = lens.copy(), np.zeros_like(w)
    for r, n in enumerate(lens):
        kept = np.arange(n)
        if n > s["limit"]:
            between = kept[s["first"]:n - s["recent"]]
            best = between[np.lexsort((between, -w[r, between]))][:s["budget"] - s["first"] - s["recent"]]
            kept = np.sort(np.concatenate([kept[:s["first"]], best, kept[n - s["recent"]:]]))
        new[r] = len(kept)
        out[r, :len(kept)] = w[r, kept]
    return {"table": None, "lens": new, "refs": None, "weights": out, "cache": None}


def exact(case, seed):
    s = prepare(case, seed)
    return {"verify": _exact_verify, "weights": _exact_weights, "evict": _exact_evict}[case["op"]](s)
