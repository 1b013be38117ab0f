"""The lists of cache slots of dsv4_sparse_mla_decode_fp4, entry for entry, and that every entry is decoded once.

The workspace begins with the slots [tokens, topk_width + window]; they are compared with oracle.combine taken through the block
table.  With queries of zero every logit is 0 and every weight exactly 1, so a head's lse is ln(keys + e^sink) but for an fp32
logarithm (2^-22 of it, and 2^-23 for the sink's exponential): one key too many or too few of 40000 is 2^-15."""
import dataclasses

import numpy as np
import pytest
import torch

import oracle
import sparse_mla_decode_combine_gb300 as pkg
import synth
from fp4_util import compare, run, to_fp4, unlisted_as_nan
from gpu_util import edge_workload, junk_workload, long_window_workload, need_gpu, small, widest_workload
from oracle import fp4

pytestmark = pytest.mark.gpu


def check(w):
    T, H, W = w.num_tokens, w.num_heads, w.topk_width + w.window
    lists, lens = oracle.combine(w.topk_idx, w.topk_lens, w.seq_lens, w.window, W)
    d = synth.to_device(dataclasses.replace(w, q=np.zeros_like(w.q)), "cuda")
    ws = pkg.workspace_for_fp4(T, H, w.topk_width, w.window)
    ws.fill_(0xA5)
    _, lse = pkg.sparse_mla_decode_fp4(**d, workspace=ws)
    slots = ws[:4 * T * W].view(torch.int32).view(T, W).cpu().numpy()
    got = lse.double().cpu().numpy()
    for t in range(T):
        p = lists[t, :lens[t]].astype(np.int64)
        row = t if w.req_idx is None else int(w.req_idx[t])
        want = w.block_table[row, p // w.page].astype(np.int64) * w.page + p % w.page
        assert np.array_equal(slots[t, :lens[t]], want), (w.name, t, np.flatnonzero(slots[t, :lens[t]] != want)[:4])
        sums = lens[t] + (np.exp(w.sink.astype(np.float64)) if w.sink is not None else np.zeros(H))
        with np.errstate(divide="ignore"):
            ref = np.log(sums)
        if lens[t] == 0:
            assert np.array_equal(got[t], w.sink if w.sink is not None else np.full(H, -np.inf))
        else:
            assert np.all(np.abs(got[t] - ref) <= 2.0 ** -22 * np.abs(ref) + 2.0 ** -22), (w.name, t, lens[t], np.exp(got[t]).max())
    assert pkg.dsv4_get_device_status() == pkg.DSV4_OK


def repeats(w):
    rows = w.topk_idx.copy()
    n = rows[:, 1::3].shape[1]
    rows[:, 1::3] = rows[:, 0::3][:, :n]
    return dataclasses.replace(w, topk_idx=rows, name=w.name + ", repeats")


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5])
def test_small_configs(n):
    need_gpu()
    check(unlisted_as_nan(to_fp4(small(n))))


@pytest.mark.parametrize("tokens,heads,topk,window,seq", [
    (1, 16, 0, 20000, 20000), (1, 16, 0, 40000, 30000), (1, 64, 2048, 128, 9000), (2, 16, 64, 0, 700), (3, 128, 1279, 100, 5000),
    (3, 128, 1280, 100, 5000), (3, 32, 1281, 100, 5000), (5, 16, 1, 63, 900), (1, 128, 0, 1, 10)])
def test_few_tokens_shared_by_many(tokens, heads, topk, window, seq):
    """A token's list is made by the CTAs that share it, the window's part by each for itself, or by the list kernel."""
    need_gpu()
    rng = np.random.default_rng(topk + window)
    seqs = [seq] + rng.integers(0, seq, tokens - 1).tolist()
    w = to_fp4(synth.make_workload(name="few", seed=98, heads=heads, req_seq_lens=seqs, topk_width=topk, window=window, sink=True))
    check(unlisted_as_nan(w))
    if topk > 3:
        check(repeats(w))


@pytest.mark.parametrize("tokens,heads", [(75, 64), (77, 64), (40, 128), (128, 128), (700, 16), (1300, 16)])
def test_runs_over_many_tokens(tokens, heads):
    """Runs of blocks that begin and end inside tokens, and runs that end between them."""
    need_gpu()
    rng = np.random.default_rng(tokens)
    seqs = rng.integers(0, 700, tokens)
    seqs[rng.random(tokens) < 0.1] = 0
    w = to_fp4(synth.make_workload(name="runs", seed=99, heads=heads, req_seq_lens=seqs, topk_width=260, window=70, sink=False))
    check(w)
    check(repeats(w))


@pytest.mark.parametrize("w", [lambda: junk_workload(64), lambda: widest_workload(16), long_window_workload,
                               lambda: edge_workload(128, True), lambda: edge_workload(32, False, window=0)],
                         ids=["junk", "widest", "long window", "edge", "no window"])
def test_rows_of_more_than_one_pass_and_junk(w):
    need_gpu()
    check(to_fp4(w()))


def far(tokens, heads, topk, window, selectable, seed=0):
    """Histories of `selectable` positions before the window, their pages drawn from a pool of 40 (positions share pages, so a
    long history costs nothing); rows name positions over all of it, its last ones and those around 2^18 among them."""
    rng = np.random.default_rng([topk, selectable, seed])
    w = to_fp4(synth.make_workload(name="pool", seed=100, heads=heads, req_seq_lens=[40 * 64] + [1] * (tokens - 1), topk_width=topk,
                                   window=window, sink=True))
    seq = selectable + window
    table = rng.integers(0, 40, (tokens, -(-seq // 64))).astype(np.int32)
    rows = np.stack([rng.choice(selectable, topk, replace=False) for _ in range(tokens)]).astype(np.int32)
    edge = [selectable - 1, 0, selectable - 2] + [v for v in range(262140, 262150) if v < selectable]
    for t in range(tokens):
        rest = rows[t][~np.isin(rows[t], edge)]
        rows[t] = rng.permutation(np.concatenate([edge, rest]))[:topk] if topk < len(edge) + len(rest) else rng.permutation(
            np.concatenate([edge, rest, np.full(topk - len(edge) - len(rest), -1)]))
    rows[:, -1] = selectable                            # in the window: dropped
    return dataclasses.replace(w, name=f"{selectable} before the window", block_table=table, topk_idx=rows,
                               seq_lens=np.full(tokens, seq, np.int32))


@pytest.mark.parametrize("tokens", [2, 90])
@pytest.mark.parametrize("topk,bitmap", [(512, 1 << 18), (1280, 1 << 18), (1281, 1 << 18), (2048, 1 << 18), (3000, 1 << 19),
                                         (8192, 1 << 20)])
@pytest.mark.parametrize("past", [-1, 0, 1, 40000])
def test_histories_around_the_bitmaps_length(tokens, topk, bitmap, past):
    """Up to `bitmap` positions before the window repeats are looked for in a bitmap, past them in a hash set from the start:
    rows of one round of loads and of several, in lists made by the decode and by the list kernel, without and with repeats."""
    need_gpu()
    w = far(tokens, 16 if tokens == 2 else 64, topk, 70, bitmap + past)
    check(w)
    check(repeats(w))


@pytest.mark.parametrize("topk", [512, 3000])
def test_far_histories_decode(topk):
    need_gpu()
    w = repeats(far(3, 64, topk, 70, 600001))
    out, lse, st = run(w)
    assert st == pkg.DSV4_OK
    compare(out, lse, fp4.decode(w), w.name)
