"""The 4-bit operators and the page operators in the order of their stream: each launch may begin while the one before it
ends, so what a call reads has to be what the kernels before it wrote, and calls on several streams must not meet."""
import numpy as np
import pytest
import torch

import sparse_mla_decode_combine_gb300 as pkg
import synth
from fp4_util import to_fp4
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def workload(tokens, heads):
    rng = np.random.default_rng(tokens)
    w = to_fp4(synth.make_workload(name=f"{tokens} x {heads}", seed=70, heads=heads, req_seq_lens=rng.integers(200, 900, tokens),
                                   topk_width=256, window=64, sink=False))
    return synth.to_device(w, "cuda")


@pytest.mark.parametrize("tokens,heads", [(1, 16), (32, 64), (90, 128)])
def test_everything_that_a_decode_reads_is_written_just_before_it(tokens, heads):
    need_gpu()
    d = workload(tokens, heads)
    names = ["q", "kv_cache", "block_table", "topk_idx", "seq_lens"]
    clean = {k: d[k].clone() for k in names}
    qs = [torch.randn(d["q"].shape, device="cuda").bfloat16() for _ in range(6)]
    want = [tuple(t.clone() for t in pkg.sparse_mla_decode_fp4(**{**d, "q": q})) for q in qs]
    torch.cuda.synchronize()
    ws = pkg.workspace_for_fp4(tokens, heads, d["topk_idx"].shape[1], d["window"])
    out = torch.empty((tokens, heads, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((tokens, heads), device="cuda")
    busy = torch.randn((3000, 3000), device="cuda")
    for late in names:                      # the input that the kernel directly before the call writes
        got = []
        for q in qs:
            for k in names:
                d[k].zero_()
            busy = (busy @ busy).clamp_(-1, 1)
            for k in [k for k in names if k != late] + [late]:
                d[k].copy_(q if k == "q" else clean[k])
            pkg.check(pkg.dsv4_sparse_mla_decode_fp4(out=out, lse=lse, workspace=ws, **d))
            got.append((out.clone(), lse.clone()))
        torch.cuda.synchronize()
        for (a, b), (x, y) in zip(got, want):
            assert torch.equal(a, x) and torch.equal(b, y), late
    assert pkg.dsv4_get_device_status() == pkg.DSV4_OK


def serve(seed, sync, stream=None):
    """Rounds of insert, fork, compact, copy and decode over one pool, each reading what the one before it wrote."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    page, blocks, R, M, H = 4, 96, 6, 8, 16
    cache = torch.zeros((2, blocks, page, 400), dtype=torch.uint8, device="cuda")
    other = torch.zeros_like(cache)
    ang = torch.rand((64, 32), generator=g, device="cuda")
    cs = torch.cat([torch.cos(ang), torch.sin(ang)], 1).contiguous()
    table = torch.arange(R * M, dtype=torch.int32, device="cuda").reshape(R, M)
    lens = torch.full((R,), 14, dtype=torch.int32, device="cuda")
    refs = torch.zeros(blocks, dtype=torch.int32, device="cuda")
    refs[:R * M] = (torch.arange(R * M, device="cuda") % M < 4).int()
    none = torch.empty((R, 0), dtype=torch.int32, device="cuda")
    ws = pkg.workspace_for_fp4(R, H, 0, 40)
    wp = pkg.workspace_for_cache_pages(R, R, blocks)
    made = []
    wait = torch.cuda.synchronize if sync else (lambda: None)
    for r in range(8):
        slots = (table[:, :4, None].long() * page + torch.arange(page, device="cuda")).reshape(R, -1)[:, :14].reshape(-1)
        slots = torch.where(torch.arange(R * 14, device="cuda") // 14 == r % R, slots, -1)     # one row's keys again
        n = len(slots)
        for layer in range(2):
            wait()
            q = rnd(n, H, 576)
            pkg.check(pkg.dsv4_qk_norm_rope_kv_insert_fp4(q, q, rnd(n, 576), torch.arange(n, device="cuda") % 64, slots, cs,
                                                          cache[layer], stream=stream))
            wait()
        parent = torch.randint(0, R, (R,), generator=g, device="cuda").int()
        t2, l2, r2 = torch.empty_like(table), torch.empty_like(lens), torch.empty_like(refs)
        pkg.check(pkg.dsv4_cache_fork_rows(cache, table, lens, refs, parent, t2, l2, r2, wp, True, stream))
        wait()
        pmap, live = torch.empty_like(refs), i32(0)
        pkg.check(pkg.dsv4_cache_compact(cache, t2, l2, r2, t2, r2, pmap, live, wp, stream))
        wait()
        src = t2[:, 0].contiguous()
        pkg.check(pkg.dsv4_cache_copy_pages(other, cache, src, src, wp, stream))
        wait()
        table, lens, refs = t2, l2, r2
        out = torch.empty((R, H, 512), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((R, H), device="cuda")
        pkg.check(pkg.dsv4_sparse_mla_decode_fp4(q[:R], cache[1], table, None, none, None, lens, 40, None, 0.05, out, lse, ws,
                                                 stream))
        wait()
        made += [out, lse, table, refs, pmap, live, cache.clone(), other.clone()]
    return made


def test_a_chain_of_calls_without_a_wait_between_them():
    need_gpu()
    want = serve(1, True)
    for _ in range(3):
        got = serve(1, False)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert not torch.isnan(want[-7]).any()
    assert pkg.dsv4_get_device_status() == pkg.DSV4_OK


def test_chains_on_three_streams_at_once():
    need_gpu()
    want = [serve(s, True) for s in (1, 2, 3)]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for s, st in zip((1, 2, 3), streams):
        with torch.cuda.stream(st):
            got.append(serve(s, False))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert pkg.dsv4_get_device_status() == pkg.DSV4_OK


@pytest.mark.parametrize("tokens,heads", [(2, 16), (90, 128)])
def test_captured_behind_a_copy_and_two_streams(tokens, heads):
    """In a graph, a call whose inputs come from a memset, from a copy and from kernels of two other streams."""
    need_gpu()
    d = workload(tokens, heads)
    H = heads
    want, wlse = (t.clone() for t in pkg.sparse_mla_decode_fp4(**d))
    clean = {k: d[k].clone() for k in ("q", "topk_idx", "kv_cache")}
    ws = pkg.workspace_for_fp4(tokens, heads, d["topk_idx"].shape[1], d["window"])
    wp = pkg.workspace_for_cache_pages(0, 0, d["kv_cache"].shape[0])
    out = torch.empty((tokens, H, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((tokens, H), device="cuda")
    moved = torch.zeros_like(d["kv_cache"])
    pages = torch.zeros(d["kv_cache"].shape[0], dtype=torch.int32, device="cuda")
    main, a, b = (torch.cuda.Stream() for _ in range(3))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=main):
        a.wait_stream(main)
        b.wait_stream(main)
        with torch.cuda.stream(a):
            d["q"].copy_(clean["q"] * 1)
        with torch.cuda.stream(b):
            pages.zero_()
            pages += torch.arange(len(pages), device="cuda").int()
            pkg.check(pkg.dsv4_cache_copy_pages(moved[None], clean["kv_cache"][None], pages, pages, wp))
        d["topk_idx"].copy_(clean["topk_idx"])
        out.zero_()
        main.wait_stream(a)
        main.wait_stream(b)
        pkg.check(pkg.dsv4_sparse_mla_decode_fp4(out=out, lse=lse, workspace=ws, **{**d, "kv_cache": moved}))
    for _ in range(3):
        for t in (d["q"], d["topk_idx"], moved, out, lse):
            t.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wlse)
    assert pkg.dsv4_get_device_status() == pkg.DSV4_OK
