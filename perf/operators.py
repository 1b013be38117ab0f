"""The 4-bit cache's operators, as a serving loop calls them: the sparse-MLA decode over a cache whose latent is
held in 4 bits, the fused norm + rotation + 4-bit insert that fills it, and the page operators (fork, compact, copy)
that manage its pages.

`own` chooses between the framework's kernels (true) and the plain form in elementary torch operations (false).  The
plain forms compute in 32 bits and round once at the end; the 4-bit quantisation runs in 64 bits, where a value next
to a rounding border is decided.

The cache entry (400 bytes): 512 E2M1 codes (element 2i in the low half of byte i), 64 BF16 rope values, 16 UE8M0
scale bytes, one for each 32 latent values.
"""
import math

import numpy as np
import torch

own = False

ENTRY = 400          # bytes of a 4-bit entry
ENTRY_FP8 = 656      # bytes of an 8-bit entry: the page operators move either
DIM, LATENT, ROPE = 576, 512, 64
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)      # magnitudes of the E2M1 codes 0..7


# --------------------------------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------------------------------
def listed():
    return [
        # one small request batch answered at once: latency is all there is
        dict(name="decode-tiny", op="decode", tokens=2, per_req=1, heads=16, seq_lo=256, seq_hi=256, topk=64, ragged=False,
             window=32, sink=False, page=64, pad=0, heavy=False),
        # an ordinary decode batch
        dict(name="decode-mid", op="decode", tokens=32, per_req=1, heads=64, seq_lo=8192, seq_hi=8192, topk=512,
             ragged=False, window=128, sink=False, page=64, pad=0, heavy=False),
        # speculative verification: two tokens a request, ragged histories and list lengths
        dict(name="decode-verify", op="decode", tokens=128, per_req=2, heads=128, seq_lo=4096, seq_hi=65536, topk=2048,
             ragged=True, window=128, sink=True, page=64, pad=0, heavy=False),
        # the largest batch: 128 heads over 2176 keys a token
        dict(name="decode-heavy", op="decode", tokens=128, per_req=1, heads=128, seq_lo=32768, seq_hi=32768, topk=2048,
             ragged=False, window=128, sink=True, page=64, pad=0, heavy=False),
        # the insert of one decode step of a large batch, a few padding tokens at its end
        dict(name="insert-decode", op="insert", tokens=128, heads=128, norm_dims=512, weights=True, slots=65536,
             max_pos=32768, pad=3, gap=0),
        # a prefill chunk of odd length, queries in rows wider than their heads
        dict(name="insert-prefill", op="insert", tokens=8191, heads=64, norm_dims=512, weights=True, slots=65536,
             max_pos=32768, pad=0, gap=64),
        # one step of beam search: rows share their prompts, every beam picks its parent anew
        dict(name="fork-beam", op="fork", groups=16, beams=4, prompt=1000, tail=500, page=64, entry=ENTRY, layers=8,
             blocks=1024, drop=0.1, share=True, children=1),
        # parallel sampling with private copies of whole prompts
        dict(name="fork-private", op="fork", groups=8, beams=1, prompt=4000, tail=200, page=64, entry=ENTRY, layers=8,
             blocks=4096, drop=0.0, share=False, children=4),
        # a small pool with a few holes
        dict(name="compact-small", op="compact", groups=8, beams=2, prompt=700, tail=200, page=64, entry=ENTRY, layers=2,
             blocks=333, live=0.5),
        # a large pool half of whose pages were freed
        dict(name="compact-large", op="compact", groups=64, beams=2, prompt=3500, tail=900, page=64, entry=ENTRY,
             layers=8, blocks=8192, live=0.6),
        # a handful of pages, as when one request is swapped in
        dict(name="copy-few", op="copy", pages=7, page=64, entry=ENTRY, layers=4, blocks=512, two_pools=False),
        # many pages into another pool, 8-bit entries
        dict(name="copy-many", op="copy", pages=1501, page=32, entry=ENTRY_FP8, layers=8, blocks=2048, two_pools=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("decode", "decode", "insert", "fork", "compact", "copy"))
    if op == "decode":
        per_req = rng.choice((1, 1, 2))
        reqs = _log(rng, 1, 128 // per_req)
        seq_hi = min(_log(rng, 48, 131072), 4_000_000 // reqs)
        return dict(op=op, tokens=reqs * per_req, per_req=per_req, heads=rng.choice((16, 32, 64, 128)),
                    seq_lo=max(per_req, seq_hi // rng.choice((1, 4, 16))), seq_hi=seq_hi, topk=_log(rng, 16, 2048),
                    ragged=rng.random() < 0.5, window=rng.choice((0, 1, 17, 32, 64, 100, 128)), sink=rng.random() < 0.5,
                    page=rng.choice((16, 32, 64, 256)), pad=rng.choice((0, 0, 1, 3)), heavy=rng.random() < 0.3)
    if op == "insert":
        return dict(op=op, tokens=_log(rng, 1, 8000), heads=rng.choice((1, 8, 16, 32, 63, 64)),
                    norm_dims=rng.choice((0, 512, 512, 576)), weights=rng.random() < 0.7, slots=rng.randrange(9000, 60000),
                    max_pos=_log(rng, 64, 32768), pad=rng.choice((0, 0, 1, 5)), gap=rng.choice((0, 8, 576)))
    page, entry = rng.choice((16, 32, 64)), rng.choice((ENTRY, ENTRY, ENTRY_FP8))
    layers = rng.choice((1, 2, 3, 5))
    if op == "fork":
        share = rng.random() < 0.6
        groups, beams = _log(rng, 1, 24), rng.choice((1, 2, 3, 4, 8)) if share else 1
        return dict(op=op, groups=groups, beams=beams, prompt=_log(rng, 16, 1500), tail=_log(rng, 1, 300), page=page,
                    entry=entry, layers=layers, blocks=16384 * 16 // page, drop=rng.choice((0.0, 0.1, 0.5)), share=share,
                    children=rng.choice((1, 2, 3)))
    if op == "compact":
        return dict(op=op, groups=_log(rng, 1, 48), beams=rng.choice((1, 2, 4)), prompt=_log(rng, 16, 2000),
                    tail=_log(rng, 1, 300), page=page, entry=entry, layers=layers, blocks=_log(rng, 300, 12000),
                    live=rng.uniform(0.05, 0.95))
    blocks = _log(rng, 64, 6000)
    return dict(op=op, pages=_log(rng, 1, min(1500, blocks // 2)), page=page, entry=entry, layers=layers, blocks=blocks,
                two_pools=rng.random() < 0.5)


# --------------------------------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------------------------------
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _quantised(latent):
    """Real (codes, scale bytes) of random latents: what a cache in use holds."""
    x = latent.double().view(-1, 16, 32)
    amax = x.abs().amax(-1)
    m, k = torch.frexp(amax / 6.0)                          # amax / 6 = m 2^k, 1/2 <= m < 1
    e = torch.where(m > 0.5, k, k - 1)
    e = torch.where(amax > 0, e, torch.zeros_like(e)).clamp(-127, 125)
    y = torch.ldexp(x, -e[..., None])
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device=x.device)
    code = torch.bucketize(y.abs(), mids)
    code = (code | (torch.signbit(y).to(code.dtype) << 3)).view(-1, LATENT).to(torch.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), (e + 127).to(torch.uint8)


def _cache(g, slots, heavy):
    """A cache whose entries are draws from a pool of quantised rows."""
    n = min(slots, 8192)
    x = torch.randn(n, LATENT, generator=g, device="cuda")
    if heavy:                                               # Student-t with three degrees of freedom
        x = x / (torch.randn(n, LATENT, 3, generator=g, device="cuda").square().mean(-1)).sqrt()
    codes, scales = _quantised(x)
    rope = torch.randn(n, ROPE, generator=g, device="cuda").bfloat16().view(torch.uint8)
    pool = torch.cat([codes, rope, scales], 1)
    out = torch.empty(slots, ENTRY, dtype=torch.uint8, device="cuda")
    for lo in range(0, slots, 1 << 20):                     # (in parts, for the index's sake)
        hi = min(slots, lo + (1 << 20))
        out[lo:hi] = pool[torch.randint(0, n, (hi - lo,), generator=g, device="cuda")]
    return out


def _prepare_decode(c, seed):
    g, r = _generator(seed), np.random.default_rng(seed)
    reqs = c["tokens"] // c["per_req"]
    pad, page, K = c["pad"], c["page"], c["topk"]
    lens = r.integers(c["seq_lo"], c["seq_hi"], size=reqs, endpoint=True)
    pages = -(-lens // page)
    table = np.full((reqs, int(pages.max())), -1, dtype=np.int32)
    perm, at = r.permutation(int(pages.sum())).astype(np.int32), 0
    for i, n in enumerate(pages):
        table[i, :n] = perm[at:at + n]
        at += n
    pos = np.concatenate([np.arange(s - c["per_req"], s) for s in lens])
    T = c["tokens"] + pad                                   # padding tokens see nothing
    seq = torch.tensor(np.concatenate([pos + 1, np.zeros(pad)]), dtype=torch.int32, device="cuda")
    req = torch.tensor(np.concatenate([np.repeat(np.arange(reqs), c["per_req"]), np.zeros(pad)]), dtype=torch.int32,
                       device="cuda")
    score = torch.rand(T, max(K, c["seq_hi"]), generator=g, device="cuda")
    score.masked_fill_(torch.arange(score.shape[1], device="cuda") >= seq[:, None], -1.0)
    best, idx = score.topk(K, dim=1)                        # distinct positions in random order
    idx = torch.where(best >= 0, idx, -1).to(torch.int32)
    n = (best >= 0).sum(1).to(torch.int32)
    lens_k = None
    if c["ragged"]:
        lens_k = torch.minimum(n, torch.randint(max(1, K // 8), K + 1, (T,), generator=g, device="cuda", dtype=torch.int32))
        idx = torch.where(torch.arange(K, device="cuda") < lens_k[:, None], idx, -1)
    H = c["heads"]
    state = dict(
        op="decode", q=torch.randn(T, H, DIM, generator=g, device="cuda").bfloat16(),
        cache=_cache(g, int(pages.sum()) * page, c["heavy"]).view(-1, page, ENTRY),
        table=torch.from_numpy(table).cuda(), req=req, topk=idx.contiguous(), topk_lens=lens_k, seq=seq,
        window=c["window"], sink=torch.randn(H, generator=g, device="cuda") if c["sink"] else None,
        scale=1.0 / math.sqrt(DIM), out=torch.empty(T, H, LATENT, dtype=torch.bfloat16, device="cuda"),
        lse=torch.empty(T, H, dtype=torch.float32, device="cuda"), workspace=None)
    if own:
        import sparse_mla_decode_combine_gb300 as pkg
        state["workspace"] = pkg.workspace_for_fp4(T, H, K, c["window"])
    return state


def _prepare_insert(c, seed):
    g = _generator(seed)
    T, H = c["tokens"], c["heads"]
    wide = torch.randn(T, H * DIM + c["gap"], generator=g, device="cuda")
    wide = (wide * torch.empty(T, 1, device="cuda").uniform_(0.1, 10.0, generator=g)).bfloat16()
    q = wide[:, :H * DIM].view(T, H, DIM)
    kv = torch.randn(T, DIM, generator=g, device="cuda") * torch.empty(T, 1, device="cuda").uniform_(0.01, 30.0, generator=g)
    slots = torch.randperm(c["slots"], generator=g, device="cuda")[:T].contiguous()
    if c["pad"]:
        slots[max(0, T - c["pad"]):] = -1
    inv = 10000.0 ** (-torch.arange(32, dtype=torch.float64, device="cuda") / 32)
    ang = torch.arange(c["max_pos"], dtype=torch.float64, device="cuda")[:, None] * inv
    w = c["weights"]
    n = c["norm_dims"]
    return dict(
        op="insert", q=q, kv=kv.bfloat16(), pos=torch.randint(0, c["max_pos"], (T,), generator=g, device="cuda"),
        slots=slots, cos_sin=torch.cat([ang.cos(), ang.sin()], 1).float().contiguous(), norm_dims=n, eps=1e-6,
        qw=torch.empty(DIM, device="cuda").uniform_(0.5, 1.5, generator=g) if w else None,
        kw=torch.empty(n, device="cuda").uniform_(0.5, 1.5, generator=g) if w and n else None,
        cache=torch.zeros(c["slots"], ENTRY, dtype=torch.uint8, device="cuda"),
        q_out=torch.empty(T, H, DIM, dtype=torch.bfloat16, device="cuda"),
        k_out=torch.empty(T, DIM, dtype=torch.bfloat16, device="cuda"))


def _rows(r, c, most):
    """Rows of a pool in use: `beams` rows a group share their prompt's full pages; at most `most` pages are taken."""
    page = c["page"]
    perm, at = r.permutation(c["blocks"]).astype(np.int32), 0
    lens, rows = [], []
    for _ in range(c["groups"]):
        prompt = int(r.integers(max(1, c["prompt"] // 2), c["prompt"] + 1))
        shared = prompt // page
        todo = [prompt + int(r.integers(1, c["tail"] + 1)) for _ in range(c["beams"])]
        if at + shared + sum(-(-n // page) - shared for n in todo) > most:
            todo = [0] * c["beams"]                         # the pool is as full as asked: the other rows are empty
        head = perm[at:at + shared] if todo[0] else perm[:0]
        at += len(head)
        for n in todo:
            own_pages = max(0, -(-n // page) - shared)
            rows.append(np.concatenate([head, perm[at:at + own_pages]]))
            at += own_pages
            lens.append(n)
    width = -(-(c["prompt"] + c["tail"]) // page) + 3       # rows have room to grow
    table = np.full((len(rows), width), -1, dtype=np.int32)
    for i, p in enumerate(rows):
        table[i, :len(p)] = p
    refs = np.bincount(table[table >= 0], minlength=c["blocks"]).astype(np.int32)
    return table, np.array(lens, dtype=np.int32), refs


def _pool(g, c):
    return torch.randint(0, 256, (c["layers"], c["blocks"], c["page"], c["entry"]), dtype=torch.uint8, generator=g,
                         device="cuda")


def _prepare_fork(c, seed):
    g, r = _generator(seed), np.random.default_rng(seed)
    table, lens, refs = _rows(r, c, c["blocks"])
    G, b = c["groups"], c["beams"]
    n = b * c["children"]
    parent = np.arange(G)[:, None] * b + r.integers(0, b, size=(G, n))
    parent = np.where(r.random((G, 1)) < c["drop"], -1, parent).reshape(-1).astype(np.int32)   # finished requests go
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    state = dict(op="fork", cache=_pool(g, c), table=dev(table), lens=dev(lens), refs=dev(refs), parent=dev(parent),
                 share=c["share"], table_out=torch.empty(G * n, table.shape[1], dtype=torch.int32, device="cuda"),
                 lens_out=torch.empty(G * n, dtype=torch.int32, device="cuda"),
                 refs_out=torch.empty(c["blocks"], dtype=torch.int32, device="cuda"), workspace=None)
    if own:
        import sparse_mla_decode_combine_gb300 as pkg
        state["workspace"] = pkg.workspace_for_cache_pages(len(lens), G * n, c["blocks"])
    return state


def _prepare_compact(c, seed):
    g, r = _generator(seed), np.random.default_rng(seed)
    table, lens, refs = _rows(r, c, max(1, int(c["blocks"] * c["live"])))
    spare = np.flatnonzero(refs == 0)                       # pages that a prefix cache, not a row, holds
    held = spare[r.random(len(spare)) < 0.5 * max(0.0, c["live"] - (refs > 0).mean())]
    refs[held] = 1
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    state = dict(op="compact", cache=_pool(g, c), table=dev(table), lens=dev(lens), refs=dev(refs),
                 table_out=torch.empty(table.shape, dtype=torch.int32, device="cuda"),
                 refs_out=torch.empty(c["blocks"], dtype=torch.int32, device="cuda"),
                 page_map=torch.empty(c["blocks"], dtype=torch.int32, device="cuda"),
                 live=torch.empty(1, dtype=torch.int32, device="cuda"), workspace=None)
    if own:
        import sparse_mla_decode_combine_gb300 as pkg
        state["workspace"] = pkg.workspace_for_cache_pages(0, 0, c["blocks"])
    return state


def _prepare_copy(c, seed):
    g, r = _generator(seed), np.random.default_rng(seed)
    n = c["pages"]
    perm = r.permutation(c["blocks"]).astype(np.int32)
    src, dst = perm[:n].copy(), perm[-n:].copy()            # one pool: sources and targets are apart
    cache = _pool(g, c)
    state = dict(op="copy", dst_cache=cache, src_cache=_pool(g, c) if c["two_pools"] else cache,
                 src=torch.from_numpy(src).cuda(), dst=torch.from_numpy(dst).cuda(), workspace=None)
    if own:
        import sparse_mla_decode_combine_gb300 as pkg
        state["workspace"] = pkg.workspace_for_cache_pages(0, 0, c["blocks"])
    return state


def prepare(case, seed):
    return {"decode": _prepare_decode, "insert": _prepare_insert, "fork": _prepare_fork, "compact": _prepare_compact,
            "copy": _prepare_copy}[case["op"]](case, seed)


# --------------------------------------------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------------------------------------------
def _dequantised(entries):
    """uint8 [..., 400] -> float32 keys [..., 576]."""
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device=entries.device)
    codes = entries[..., :256]
    latent = torch.stack([grid[(codes & 15).long()], grid[(codes >> 4).long()]], -1).flatten(-2)
    scale = torch.exp2(entries[..., 384:].float() - 127.0)
    latent = (latent.unflatten(-1, (16, 32)) * scale[..., None]).flatten(-2)
    rope = entries[..., 256:384].contiguous().view(torch.bfloat16).float()
    return torch.cat([latent, rope], -1)


def _decode(s):
    topk, W = s["topk"].long(), s["window"]
    T, K = topk.shape
    dev = topk.device
    pos = s["seq"].long() - 1
    lo = (pos - W + 1).clamp(min=0)
    n = torch.full_like(pos, K) if s["topk_lens"] is None else s["topk_lens"].long().clamp(0, K)
    ok = (torch.arange(K, device=dev) < n[:, None]) & (topk >= 0) & (topk < lo[:, None])
    srt, order = torch.where(ok, topk, -1).sort(dim=1, stable=True)          # repeats: the first one stays
    fresh = torch.cat([torch.ones(T, 1, dtype=torch.bool, device=dev), srt[:, 1:] != srt[:, :-1]], 1)
    ok &= torch.zeros_like(ok).scatter(1, order, fresh)
    win = lo[:, None] + torch.arange(W, device=dev)
    p = torch.cat([topk, win], 1)
    ok = torch.cat([ok, win <= pos[:, None]], 1)
    p = torch.where(ok, p, 0)
    page = s["cache"].shape[1]
    block = s["table"][s["req"].long()[:, None], p // page].long()
    k = _dequantised(s["cache"][torch.where(ok, block, 0), p % page])
    logits = torch.matmul(s["q"].float(), k.transpose(1, 2)) * s["scale"]
    logits = logits.masked_fill(~ok[:, None, :], -torch.inf)
    m = logits.amax(-1, keepdim=True)
    if s["sink"] is not None:
        m = torch.maximum(m, s["sink"][None, :, None])
    m = torch.where(m == -torch.inf, 0.0, m)
    e = torch.exp(logits - m)
    z = e.sum(-1, keepdim=True)
    if s["sink"] is not None:
        z = z + torch.exp(s["sink"][None, :, None] - m)
    out = torch.matmul(e, k[..., :LATENT]) / torch.where(z > 0, z, 1.0)
    return {"out": out.bfloat16(), "lse": (m + torch.log(z)).squeeze(-1)}


def _rotated(x, c, s):
    """GPT-J rotation of the pairs of the last 64 dims."""
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)


def _insert(s):
    q, n = s["q"].float(), s["norm_dims"]
    cs = s["cos_sin"][s["pos"]]
    c, sn = cs[:, :32], cs[:, 32:]
    q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + s["eps"])
    if s["qw"] is not None:
        q = q * s["qw"]
    q_out = torch.cat([q[..., :LATENT], _rotated(q[..., LATENT:], c[:, None], sn[:, None])], -1).bfloat16()
    k = s["kv"].double()                                    # values next to a rounding border: 64 bits
    if n:
        k = torch.cat([k[:, :n] / (k[:, :n].square().mean(-1, keepdim=True) + s["eps"]).sqrt(), k[:, n:]], 1)
        if s["kw"] is not None:
            k = torch.cat([k[:, :n] * s["kw"].double(), k[:, n:]], 1)
    codes, scales = _quantised(k[:, :LATENT])
    rope = _rotated(k[:, LATENT:], c.double(), sn.double()).bfloat16()
    entry = torch.cat([codes, rope.view(torch.uint8), scales], 1)
    live = s["slots"] >= 0
    s["cache"][s["slots"][live]] = entry[live]
    return {"q": q_out, "k": _dequantised(entry).bfloat16()}


def _copied(dst_cache, src_cache, src, dst, entries=None):
    """Pages src -> dst in every layer; of each page the first `entries` entries."""
    new = src_cache[:, src]
    if entries is not None:
        within = torch.arange(new.shape[2], device=new.device) < entries[:, None]
        new = torch.where(within[None, :, :, None], new, dst_cache[:, dst])
    dst_cache[:, dst] = new


def _fork(s):
    table, lens, refs, parent = s["table"], s["lens"], s["refs"], s["parent"].long()
    page, M, dev = s["cache"].shape[2], table.shape[1], table.device
    there = parent >= 0
    pc = parent.clamp(min=0)
    n = torch.where(there, lens[pc], 0).long()
    j = torch.arange(M, device=dev)
    rows = table[pc].long()
    used = j < ((n + page - 1) // page)[:, None]
    shared = (j < (n // page)[:, None]) & s["share"]
    me = torch.arange(parent.numel(), device=dev)
    first = torch.full((table.shape[0],), parent.numel(), dtype=torch.long, device=dev)
    first = first.scatter_reduce(0, pc[there], me[there], "amin")
    keeps = (first[pc] == me)[:, None] & (refs[rows.clamp(min=0)] == 1) & used & ~shared
    need = used & ~shared & ~keeps
    free = (refs != 0).sort(stable=True).indices            # the free pages first, lowest first
    new = free[(need.flatten().cumsum(0) - 1).clamp(min=0)].view(need.shape)
    out = torch.where(need, new, torch.where(used, rows, -1))
    old = j < ((lens.long() + page - 1) // page)[:, None]
    refs_out = refs.long().scatter_add(0, table[old].long(), torch.full_like(table[old].long(), -1))
    refs_out = refs_out.scatter_add(0, out[used], torch.ones_like(out[used]))
    entries = (n[:, None] - j * page).clamp(max=page)
    _copied(s["cache"], s["cache"], rows[need], new[need], entries[need])
    return {"table": out.int(), "lens": n.int(), "refs": refs_out.int(), "cache": s["cache"]}


def _compact(s):
    refs, table, page = s["refs"], s["table"], s["cache"].shape[2]
    live = refs > 0
    count = live.sum()
    ids = torch.arange(refs.numel(), device=refs.device)
    src, dst = ids[live & (ids >= count)], ids[~live & (ids < count)]
    to = torch.where(live, ids, -1)
    to[src] = dst
    used = torch.arange(table.shape[1], device=refs.device) < ((s["lens"] + page - 1) // page)[:, None]
    out = torch.where(used, to[table.clamp(min=0).long()], -1)
    refs_out = torch.where(ids < count, refs, 0)
    refs_out[dst] = refs[src]
    _copied(s["cache"], s["cache"], src, dst)
    return {"table": out.int(), "refs": refs_out, "map": to.int(), "live": count.view(1).int(), "cache": s["cache"]}


def _copy(s):
    _copied(s["dst_cache"], s["src_cache"], s["src"].long(), s["dst"].long())
    return {"cache": s["dst_cache"]}


def run(state):
    s = state
    if own:
        import sparse_mla_decode_combine_gb300 as pkg
        if s["op"] == "decode":
            pkg.check(pkg.dsv4_sparse_mla_decode_fp4(s["q"], s["cache"], s["table"], s["req"], s["topk"], s["topk_lens"],
                                                     s["seq"], s["window"], s["sink"], s["scale"], s["out"], s["lse"],
                                                     s["workspace"]))
            return {"out": s["out"], "lse": s["lse"]}
        if s["op"] == "insert":
            pkg.check(pkg.dsv4_qk_norm_rope_kv_insert_fp4(s["q"], s["q_out"], s["kv"], s["pos"], s["slots"], s["cos_sin"],
                                                          s["cache"], s["k_out"], s["qw"], s["kw"], s["norm_dims"],
                                                          s["eps"]))
            return {"q": s["q_out"], "k": s["k_out"]}
        if s["op"] == "fork":
            pkg.check(pkg.dsv4_cache_fork_rows(s["cache"], s["table"], s["lens"], s["refs"], s["parent"], s["table_out"],
                                               s["lens_out"], s["refs_out"], s["workspace"], s["share"]))
            return {"table": s["table_out"], "lens": s["lens_out"], "refs": s["refs_out"], "cache": s["cache"]}
        if s["op"] == "compact":
            pkg.check(pkg.dsv4_cache_compact(s["cache"], s["table"], s["lens"], s["refs"], s["table_out"], s["refs_out"],
                                             s["page_map"], s["live"], s["workspace"]))
            return {"table": s["table_out"], "refs": s["refs_out"], "map": s["page_map"], "live": s["live"],
                    "cache": s["cache"]}
        pkg.check(pkg.dsv4_cache_copy_pages(s["dst_cache"], s["src_cache"], s["src"], s["dst"], s["workspace"]))
        return {"cache": s["dst_cache"]}
    return {"decode": _decode, "insert": _insert, "fork": _fork, "compact": _compact, "copy": _copy}[s["op"]](s)


# --------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "decode":
        T, H = c["tokens"] + c["pad"], c["heads"]
        seq = (c["seq_lo"] + c["seq_hi"]) / 2
        win = min(c["window"], seq)
        picks = c["topk"] * (9 / 16 if c["ragged"] else 1.0)
        picks = min(picks * max(0.0, 1 - win / seq) if c["topk"] < seq else seq, max(0.0, seq - win))
        keys = c["tokens"] * (picks + win)
        return {"bytes": keys * ENTRY + T * H * (2 * DIM + 2 * LATENT + 4) + 4 * T * c["topk"],
                "flops": 2 * keys * H * (DIM + LATENT)}
    if c["op"] == "insert":
        T, H = c["tokens"], c["heads"]
        return {"bytes": T * (H * 4 * DIM + 2 * DIM + ENTRY + 2 * DIM + 256 + 16), "flops": T * (H * 5 * DIM + 12 * DIM)}
    page_bytes = c["page"] * c["entry"] * c["layers"]
    if c["op"] == "copy":
        return {"bytes": 2 * c["pages"] * page_bytes, "flops": 0}
    rows = c["groups"] * c["beams"]
    length = 0.75 * c["prompt"] + 0.5 * c["tail"]
    width = -(-(c["prompt"] + c["tail"]) // c["page"]) + 3
    if c["op"] == "fork":
        b = c["beams"]
        kids = rows * c["children"]
        firsts = rows * (1 - (1 - 1 / b) ** (b * c["children"]))     # children that keep their parent's last page
        moved = (kids - firsts) * (0.5 * page_bytes if c["share"] else length / c["page"] * page_bytes)
        return {"bytes": 2 * (1 - c["drop"]) * moved + 4 * ((rows + kids) * width + 2 * c["blocks"]), "flops": 0}
    pages = c["groups"] * (0.75 * c["prompt"] / c["page"] + c["beams"] * (0.5 * c["tail"] / c["page"] + 0.5))
    share = min(c["live"], pages / c["blocks"])
    share += (1 - share) * 0.5 * (c["live"] - share)
    return {"bytes": 2 * share * (1 - share) * c["blocks"] * page_bytes + 4 * (2 * rows * width + 3 * c["blocks"]), "flops": 0}


# --------------------------------------------------------------------------------------------------------------
# the operators from their definitions, in 64 bits
# --------------------------------------------------------------------------------------------------------------
def _exact_key(raw):
    """uint8 numpy [n, 400] -> float64 keys [n, 576], byte by byte from the format."""
    value = np.array([(-1.0 if code & 8 else 1.0) * (0.5 * (code & 1) if (code >> 1) & 3 == 0 else
                      (1 + 0.5 * (code & 1)) * 2.0 ** (((code >> 1) & 3) - 1)) for code in range(16)])
    key = np.empty((raw.shape[0], DIM))
    key[:, 0:LATENT:2] = value[raw[:, :256] & 15]
    key[:, 1:LATENT:2] = value[raw[:, :256] >> 4]
    for b in range(16):
        key[:, 32 * b:32 * b + 32] *= np.ldexp(1.0, raw[:, 384 + b].astype(np.int64) - 127)[:, None]
    bits = raw[:, 256:384].copy().view("<u2").astype(np.uint32) << 16
    key[:, LATENT:] = bits.view(np.float32)
    return key


def _exact_decode(s):
    topk, seq, req, table = (s[k].cpu().numpy() for k in ("topk", "seq", "req", "table"))
    lens = None if s["topk_lens"] is None else s["topk_lens"].cpu().numpy()
    sink = None if s["sink"] is None else s["sink"].double()
    T, H, page = len(seq), s["q"].shape[1], s["cache"].shape[1]
    out = torch.zeros(T, H, LATENT, dtype=torch.float64, device="cuda")
    lse = torch.full((T, H), -torch.inf, dtype=torch.float64, device="cuda")
    for t in range(T):
        pos = int(seq[t]) - 1
        lo = max(0, pos - s["window"] + 1)
        picks = topk[t] if lens is None else topk[t, :lens[t]]
        picks = list(dict.fromkeys(int(p) for p in picks if 0 <= p < lo)) + list(range(lo, pos + 1))
        z = torch.zeros(H, 0, dtype=torch.float64, device="cuda")
        if picks:
            p = np.array(picks)
            block = torch.from_numpy(table[req[t], p // page].astype(np.int64)).cuda()
            key = torch.from_numpy(_exact_key(s["cache"][block, torch.from_numpy(p % page).cuda()].cpu().numpy())).cuda()
            z = (s["q"][t].double() @ key.T) * s["scale"]
        every = z if sink is None else torch.cat([z, sink[:, None]], 1)
        if every.shape[1]:
            lse[t] = torch.logsumexp(every, 1)
        if picks:
            out[t] = torch.exp(z - lse[t][:, None]) @ key[:, :LATENT]
    return {"out": out, "lse": lse}


def _exact_insert(s):
    kv, pos, cs = (s[k].double().cpu().numpy() for k in ("kv", "pos", "cos_sin"))
    n, eps, c, sn = s["norm_dims"], s["eps"], cs[pos.astype(int), :32], cs[pos.astype(int), 32:]
    if n:
        kv[:, :n] /= np.sqrt(np.mean(kv[:, :n] ** 2, axis=1, keepdims=True) + eps)
        if s["kw"] is not None:
            kv[:, :n] *= s["kw"].double().cpu().numpy()
    key = np.empty_like(kv)
    key[:, LATENT::2] = kv[:, LATENT::2] * c - kv[:, LATENT + 1::2] * sn
    key[:, LATENT + 1::2] = kv[:, LATENT::2] * sn + kv[:, LATENT + 1::2] * c
    for b in range(16):
        x = kv[:, 32 * b:32 * b + 32]
        amax = np.abs(x).max(axis=1, keepdims=True)
        e = np.full(amax.shape, -127)
        while np.any(small := (6.0 * np.ldexp(1.0, e) < amax) & (e < 125)):
            e[small] += 1
        e[amax == 0] = 0
        y = np.abs(x) * np.ldexp(1.0, -e)
        step = np.where(y < 2, 0.5, np.where(y < 4, 1.0, 2.0))               # the grid's step in the value's binade
        key[:, 32 * b:32 * b + 32] = np.copysign(np.minimum(np.rint(y / step) * step, 6.0), x) * np.ldexp(1.0, e)
    q = s["q"].double()
    q = q / torch.sqrt((q ** 2).sum(-1, keepdim=True) / DIM + eps)
    if s["qw"] is not None:
        q = q * s["qw"].double()
    c, sn = torch.from_numpy(c).cuda()[:, None], torch.from_numpy(sn).cuda()[:, None]
    turned = torch.view_as_real(torch.view_as_complex(q[..., LATENT:].unflatten(-1, (32, 2)).contiguous())
                                * torch.complex(c, sn)).flatten(-2)
    return {"q": torch.cat([q[..., :LATENT], turned], -1), "k": key}


def exact(case, seed):
    # the page operators return whole numbers alone
    if case["op"] not in ("decode", "insert"):
        return None
    s = prepare(case, seed)
    return _exact_decode(s) if case["op"] == "decode" else _exact_insert(s)
