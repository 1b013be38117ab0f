"""dsv4_sparse_mla_decode_fp4 on the GPU against the fp64 oracle (tolerances: fp4_util.compare)."""
import dataclasses

import numpy as np
import pytest
import torch

import sparse_mla_decode_combine_gb300 as pkg
import synth
from fp4_util import compare, run, to_fp4, unlisted_as_nan
from gpu_util import edge_workload, junk_workload, long_window_workload, need_gpu, small, widest_workload
from oracle import fp4

pytestmark = pytest.mark.gpu


def check(w, tokens=None, status=pkg.DSV4_OK, **over):
    out, lse, st = run(w, **over)
    assert st == status
    idx = list(range(w.num_tokens)) if tokens is None else tokens
    return compare(out[idx], lse[idx], fp4.decode(w, idx), w.name)


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5])
def test_small_configs(n):
    need_gpu()
    check(to_fp4(small(n)))


@pytest.mark.parametrize("heads", [16, 32, 64, 128])
@pytest.mark.parametrize("sink", [False, True])
def test_edge_lengths(heads, sink):
    """Empty, one-key and window-only tokens, lists that end inside a tile; every unlisted entry is NaN."""
    need_gpu()
    check(unlisted_as_nan(to_fp4(edge_workload(heads, sink))))


@pytest.mark.parametrize("heads", [16, 64, 128])
def test_only_empty_tokens(heads):
    need_gpu()
    w = to_fp4(edge_workload(heads, False, seqs=(0, 0, 0)))
    out, lse, st = run(w)
    assert st == pkg.DSV4_OK and not out.any() and bool(torch.isneginf(lse).all())


@pytest.mark.parametrize("seqs,topk,window", [((1,), 1, 0), ((1, 2, 3), 2, 1), ((127, 128, 129, 255, 256, 257), 300, 0),
                                              ((96, 97, 193), 0, 97), ((500,), 0, 1), ((1000,) * 3, 33, 256)])
@pytest.mark.parametrize("heads", [32, 128])
def test_list_lengths(seqs, topk, window, heads):
    need_gpu()
    check(unlisted_as_nan(to_fp4(edge_workload(heads, True, window=window, seqs=seqs, topk_width=topk, seed=len(seqs)))))


def test_nothing_selectable():
    """topk_width 0 and window 0: no key for any token."""
    need_gpu()
    w = to_fp4(edge_workload(64, True, window=0, seqs=(5, 0), topk_width=0))
    out, lse, st = run(w)
    assert st == pkg.DSV4_OK and not out.any() and np.array_equal(lse.cpu().numpy(), np.tile(w.sink, (2, 1)))


@pytest.mark.parametrize("heads", [16, 64, 128])
def test_junk_rows(heads):
    need_gpu()
    check(to_fp4(junk_workload(heads)))


@pytest.mark.parametrize("heads", [64, 128])
def test_widest_rows(heads):
    need_gpu()
    check(to_fp4(widest_workload(heads)))


def test_long_window():
    need_gpu()
    check(to_fp4(long_window_workload()))


@pytest.mark.parametrize("page", [1, 16, 48, 256])
def test_page_sizes(page):
    need_gpu()
    check(to_fp4(synth.make_workload(name=f"page {page}", seed=8, heads=64, req_seq_lens=[700, 33, 411], topk_width=150,
                                     window=40, sink=False, page=page, spare_pages=3)))


@pytest.mark.parametrize("heads", [16, 128])
def test_scales_far_apart(heads):
    """Blocks whose scales lie 2^40 apart: the products stay exact, the softmax is nearly one-hot."""
    need_gpu()
    check(to_fp4(synth.make_workload(name="spread", seed=9, heads=heads, req_seq_lens=[300, 80], topk_width=100, window=20,
                                     sink=True), spread=20))


def test_every_code_and_scale_byte_is_exact():
    """One key a token: the output is that key's latent, exactly, for every code under scale bytes over the BF16 range."""
    need_gpu()
    scales = np.array([0, 1, 2, 60, 100, 126, 127, 128, 129, 130, 140, 200, 250, 251, 252, 127])
    n = 16
    w = to_fp4(edge_workload(16, False, window=1, seqs=(1,) * n, topk_width=0))
    cache = w.kv_cache.copy()
    for t in range(n):
        e = cache[w.block_table[t, 0], 0]
        code = (np.arange(512) + t) % 16
        e[:256] = code[0::2] | (code[1::2] << 4)
        e[256:384] = 0
        e[384:] = np.roll(scales, t)
    w = dataclasses.replace(w, kv_cache=cache, q=np.zeros_like(w.q))
    out, lse, _ = run(w)
    want = np.stack([fp4.dequant(cache[w.block_table[t, 0], 0])[0, :512] for t in range(n)])
    got = out.double().cpu().numpy()
    assert np.array_equal(got, np.repeat(want[:, None], 16, axis=1)) and not lse.any()


def test_values_past_bf16_and_the_nan_scale():
    """6 * 2^127 has no finite BF16; scale byte 255 is NaN: they show in the dims they belong to and no other."""
    need_gpu()
    w = to_fp4(edge_workload(16, False, window=1, seqs=(1, 1), topk_width=0))
    cache = w.kv_cache.copy()
    for t, byte in enumerate((254, 255)):
        e = cache[w.block_table[t, 0], 0]
        e[:256], e[256:384], e[384:] = 0x77, 0, 127
        e[384 + 3] = byte
    w = dataclasses.replace(w, kv_cache=cache, q=np.zeros_like(w.q))
    d = {**synth.to_device(w, "cuda"), "softmax_scale": 0.0}
    out, _, _ = run(w, **{k: d[k] for k in ("softmax_scale",)})
    o = out.float().cpu().numpy()[:, 0]
    other = np.r_[0:96, 128:512]
    # 0 * inf and 0 * NaN reach the logit, so the whole token is NaN where the key holds either
    assert np.isnan(o[:, 96:128]).all() and (np.isnan(o[:, other]) | (o[:, other] == 6)).all()


@pytest.mark.parametrize("heads", [16, 64, 128])
def test_padded_batch_and_strided_queries(heads):
    """Queries in wider rows, table rows in a wider table, padding tokens (length 0) at the end with row 0 of the table."""
    need_gpu()
    w = to_fp4(synth.make_workload(name="padded", seed=12, heads=heads, req_seq_lens=[500, 0, 260, 0, 0], topk_width=130,
                                   window=16, sink=False))
    d = synth.to_device(w, "cuda")
    T = w.num_tokens
    wide = torch.full((T, heads * 576 + 24), 9.0, dtype=torch.bfloat16, device="cuda")
    q = wide[:, :heads * 576].view(T, heads, 576)
    q.copy_(d["q"])
    table = torch.full((T, w.max_blocks + 5), -3, dtype=torch.int32, device="cuda")[:, :w.max_blocks]
    table.copy_(d["block_table"])
    topk = torch.full((T, w.topk_width + 3), 7, dtype=torch.int32, device="cuda")[:, :w.topk_width]
    topk.copy_(d["topk_idx"])
    check(w, q=q, block_table=table, topk_idx=topk)


def test_slots_past_32_bit_offsets():
    """A cache of more than 2^32 bytes whose pages in use lie at its end."""
    need_gpu()
    w = to_fp4(synth.make_workload(name="far", seed=14, heads=64, req_seq_lens=[300, 900], topk_width=200, window=32,
                                   sink=False))
    n = (1 << 32) // (64 * 400) + 200
    cache = torch.empty((n, 64, 400), dtype=torch.uint8, device="cuda")
    off = n - w.num_blocks
    cache[off:] = torch.from_numpy(w.kv_cache).cuda()
    table = torch.from_numpy(np.where(w.block_table >= 0, w.block_table + off, -1).astype(np.int32)).cuda()
    check(w, kv_cache=cache, block_table=table)


def test_bad_pages_and_rows_are_left_out():
    need_gpu()
    w = to_fp4(synth.make_workload(name="bad", seed=15, heads=64, req_seq_lens=[400, 300, 200], topk_width=100, window=20,
                                   sink=True))
    table = w.block_table.copy()
    table[0, 1], table[1, 0] = w.num_blocks, -1
    w = dataclasses.replace(w, block_table=table, req_idx=np.array([0, 1, 3], np.int32))
    check(w, status=pkg.DSV4_ERR_BAD_INDEX)


def test_infinite_sinks():
    need_gpu()
    w = to_fp4(edge_workload(16, True))
    sink = w.sink.copy()
    sink[3], sink[5] = -np.inf, 80.0
    check(dataclasses.replace(w, sink=sink))


def test_without_lse_and_without_lens():
    need_gpu()
    w = to_fp4(small(2))
    d = synth.to_device(w, "cuda")
    out = torch.empty((w.num_tokens, w.num_heads, 512), dtype=torch.bfloat16, device="cuda")
    ws = pkg.workspace_for_fp4(w.num_tokens, w.num_heads, w.topk_width, w.window)
    pkg.check(pkg.dsv4_sparse_mla_decode_fp4(out=out, lse=None, workspace=ws, **d))
    torch.cuda.synchronize()
    compare(out, run(w)[1], fp4.decode(w))


@pytest.mark.parametrize("n", [2, 4])
def test_captured_and_replayed_on_another_stream(n):
    """Two graphs with a workspace each, replayed at the same time with new inputs in place."""
    need_gpu()
    ws = [to_fp4(small(n), seed=s) for s in (1, 2)]
    states, graphs = [], []
    for w in ws:
        d = synth.to_device(w, "cuda")
        out, lse = pkg.sparse_mla_decode_fp4(**d)          # (the first call on a device comes before a capture)
        work = pkg.workspace_for_fp4(w.num_tokens, w.num_heads, w.topk_width, w.window)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            pkg.check(pkg.dsv4_sparse_mla_decode_fp4(out=out, lse=lse, workspace=work, **d))
        states.append((d, out, lse, s))
        graphs.append(g)
    for r in range(2):
        for w, (d, out, lse, s) in zip(ws, states):
            out.fill_(float("nan"))
            d["q"].copy_(torch.from_numpy(w.q.view(np.int16)).view(torch.bfloat16).cuda() * (1 + r))
        torch.cuda.synchronize()
        for g, (_, _, _, s) in zip(graphs, states):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for w, (d, out, lse, _) in zip(ws, states):
            q = d["q"].view(torch.int16).cpu().numpy().view(np.uint16)
            compare(out, lse, fp4.decode(dataclasses.replace(w, q=q)), f"replay {r}")


def test_same_call_twice_is_the_same():
    need_gpu()
    w = to_fp4(small(4))
    (a, la, _), (b, lb, _) = run(w), run(w, stream=torch.cuda.Stream())
    assert torch.equal(a, b) and torch.equal(la, lb)


def test_many_units_are_the_same_every_time():
    """256 units of up to 700 keys, several to a CTA and split between CTAs: twenty calls give the same bits."""
    need_gpu()
    rng = np.random.default_rng(90)
    w = to_fp4(synth.make_workload(name="many", seed=91, heads=128, req_seq_lens=rng.integers(1, 1500, 128), topk_width=600,
                                   window=100, sink=True))
    d = synth.to_device(w, "cuda")
    a, la = pkg.sparse_mla_decode_fp4(**d)
    for _ in range(20):
        b, lb = pkg.sparse_mla_decode_fp4(**d)
        assert torch.equal(a, b) and torch.equal(la, lb)
    compare(a[::17], la[::17], fp4.decode(w, list(range(0, 128, 17))))


@pytest.mark.parametrize("tokens,heads", [(1, 16), (75, 64), (77, 64), (40, 128), (1300, 16)])
def test_numbers_of_units(tokens, heads):
    """Few units (shared evenly), more than half as many as multiprocessors (equal runs of blocks), and so many that runs
    end between units; some tokens are empty."""
    need_gpu()
    rng = np.random.default_rng(tokens)
    seqs = rng.integers(0, 400, tokens)
    seqs[rng.random(tokens) < 0.1] = 0
    if tokens == 1:
        seqs[:] = 390
    w = to_fp4(synth.make_workload(name=f"{tokens} tokens", seed=92, heads=heads, req_seq_lens=seqs, topk_width=260, window=70,
                                   sink=False))
    check(w, sorted(set(rng.integers(0, tokens, 60).tolist()) | {0, tokens - 1}))


@pytest.mark.parametrize("tokens,heads,topk,window,seq", [(1, 16, 0, 20000, 20000), (1, 64, 2048, 128, 9000), (3, 128, 1280, 100, 5000),
                                                         (3, 32, 1281, 100, 5000), (2, 16, 0, 1024, 900)])
def test_few_tokens_shared_by_many(tokens, heads, topk, window, seq):
    """One to three tokens, each shared by up to all multiprocessors: parts without keys, long windows, rows of one round of
    loads and of more, with and without repeats."""
    need_gpu()
    rng = np.random.default_rng(topk)
    seqs = [seq] + rng.integers(0, seq, tokens - 1).tolist()
    w = to_fp4(synth.make_workload(name="few", seed=94, heads=heads, req_seq_lens=seqs, topk_width=topk, window=window, sink=True))
    check(w)
    if topk:
        rows = w.topk_idx.copy()
        rows[:, 1::3] = rows[:, 0::3][:, :rows[:, 1::3].shape[1]]      # every third entry again
        check(dataclasses.replace(w, topk_idx=rows))


def test_logits_far_above_the_first_keys():
    """Later keys' logits exceed the references, which are the first key's, by far more than the range that is left to
    them, again and again: the references rise and what was summed falls."""
    need_gpu()
    w = synth.make_workload(name="rising", seed=93, heads=64, req_seq_lens=[900, 500], topk_width=0, window=600, sink=True)
    w = to_fp4(w)
    cache = w.kv_cache.copy()
    for r in range(2):                                              # the rope part grows with the position
        for pos in range(int(w.seq_lens[r])):
            e = cache[w.block_table[r, pos // 64], pos % 64]
            e[256:384] = synth.bf16_bits(np.full(64, 2.0 ** (pos / 100.0))).view(np.uint8)
    q = w.q.copy()
    q[..., 512:] = synth.bf16_bits(np.full(64, 1.0))[0]
    w = dataclasses.replace(w, kv_cache=cache, q=q, softmax_scale=1.0)
    check(w)


def test_one_key_has_nearly_all_the_weight():
    """With few tokens the output is divided by the sum of the weights as they were rounded for the product, so the rounding d
    (2^-8 at most) of the one key's weight cancels: what is left of it is d times the other keys' share e of all weight, times
    the distance of the values, 2 V, and the same again for their own roundings; then fp32's sums (2^-18 V) and the output's
    own rounding, 2^-8 of the value."""
    need_gpu()
    w = to_fp4(synth.make_workload(name="peak", seed=95, heads=16, req_seq_lens=[300, 40], topk_width=0, window=300, sink=False))
    cache = w.kv_cache.copy()
    cache[..., 256:384] = 0
    for r in range(2):
        cache[w.block_table[r, 0], 20, 256:384] = synth.bf16_bits(np.full(64, 0.25)).view(np.uint8)
    q = np.zeros_like(w.q)
    q[..., 512:] = synth.bf16_bits(0.8 + 0.05 * np.arange(16))[None, :, None]      # logits 12.8 to 24.8, all others 0
    w = dataclasses.replace(w, kv_cache=cache, q=q, softmax_scale=1.0)
    ref = fp4.decode(w)
    out, lse, _ = run(w)
    compare(out, lse, ref)
    V = np.abs(fp4.dequant(cache)[:, :512]).max()
    tol = 2.0 ** -8 * np.abs(ref[0]) + (4 * 300 * np.exp(-12.7) * 2.0 ** -8 + 2.0 ** -18) * V
    assert np.all(np.abs(out.double().cpu().numpy() - ref[0]) <= tol)


def test_refusals():
    need_gpu()
    size = pkg.dsv4_sparse_mla_decode_fp4_workspace_size
    assert size(1 << 30, 128, 0, 0) == 0 and size(1 << 20, 16, 8192, 1 << 20) == 0      # more blocks than 2^31 - 1
    assert size(0, 16, 0, 0) > 0 and size(4, 64, 512, 128) >= 4 * 4 * 640 and size(2, 64, 0, 8193) > 0
    w = to_fp4(small(1))
    d = synth.to_device(w, "cuda")
    ws = pkg.workspace_for_fp4(w.num_tokens, w.num_heads, w.topk_width, w.window)
    out = torch.empty((w.num_tokens, w.num_heads, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((w.num_tokens, w.num_heads), device="cuda")
    call = lambda **k: pkg.dsv4_sparse_mla_decode_fp4(**{**d, "out": out, "lse": lse, "workspace": ws, **k})  # noqa: E731
    assert call(workspace=ws[:-256]) == pkg.DSV4_ERR_INVALID_ARG
    assert call(workspace=torch.empty(ws.numel() + 16, dtype=torch.uint8, device="cuda")[16:]) == pkg.DSV4_ERR_INVALID_ARG
    assert call(softmax_scale=float("inf")) == pkg.DSV4_ERR_INVALID_ARG
    assert call(window=-1) == pkg.DSV4_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        call(kv_cache=torch.zeros((4, 64, 656), dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        call(seq_lens=d["seq_lens"].cpu())
    with pytest.raises(ValueError):
        call(out=out[:, :8])
    with pytest.raises(ValueError):
        call(seq_lens=d["seq_lens"][:1])
    with pytest.raises(TypeError):
        call(q=d["q"].half())
    with pytest.raises(ValueError):
        call(workspace=torch.empty((ws.numel() // 16, 32), dtype=torch.uint8, device="cuda")[:, :16])
