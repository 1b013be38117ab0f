"""The keys' attention weights on the GPU against the oracle (oracle/serving.py).

Queries and dequantised keys are exact in BF16, so what rounds is
  a logit:    an fp32 sum of 576 exact products, at most 640 roundings of the sum of magnitudes, each 2^-23 at most (the tensor
              core may truncate), and its product with the scale less the lse, one rounding each: 642 * 2^-23 times
              |q| . |k| scale + |lse|, relative to the weight;
  a weight:   the exponential, 2^-20, and the sum over up to 128 heads, 128 * 2^-24 = 2^-17, of the weight;
  the table:  one rounding for each token that is added, 2^-24 of the total.
"""
import dataclasses

import numpy as np
import pytest
import torch

import oracle
import sparse_mla_decode_combine_gb300 as pkg
import synth
from fp4_util import to_fp4
from gpu_util import edge_workload, junk_workload, need_gpu
from oracle import fp4, serving

pytestmark = pytest.mark.gpu


def lse_of(w):
    return np.asarray(fp4.decode(w)[1] if w.kv_cache.shape[2] == 400 else oracle.sparse_mla_decode(w)[1], np.float32)


def run(w, lse, table, stream=None, gap=0, **over):
    d = {**synth.to_device(w, "cuda"), **over}
    d.pop("sink", None)
    R, W = table.shape
    full = torch.full((R + 2, W + gap), 7.0, device="cuda")
    weights = full[1:-1, :W]
    weights.copy_(torch.from_numpy(table))
    ws = pkg.workspace_for_key_weights(w.num_tokens, w.num_heads, w.topk_width, w.window)
    ws.fill_(0xA5)
    lse_d = torch.from_numpy(np.ascontiguousarray(lse, np.float32)).cuda()
    torch.cuda.synchronize()
    pkg.dsv4_get_device_status()
    pkg.check(pkg.dsv4_sparse_mla_key_weights(lse=lse_d, weights=weights, workspace=ws, stream=stream, **d), "key weights")
    torch.cuda.synchronize()
    status = pkg.dsv4_get_device_status()
    f = full.cpu().numpy()
    assert np.all(f[[0, -1]] == 7) and np.all(f[:, W:] == 7)
    return f[1:-1, :W], status


def start_table(w, seed=3):
    rng = np.random.default_rng(seed)
    return np.exp(rng.standard_normal((len(w.block_table), w.block_table.shape[1] * w.page)) - 3).astype(np.float32)


def check(w, lse=None, table=None, **kw):
    lse = lse_of(w) if lse is None else lse
    table = start_table(w) if table is None else table
    got, status = run(w, lse, table, **kw)
    want, bound, adds, bad = serving.key_weights(w, lse, table)
    assert status == (pkg.DSV4_ERR_BAD_INDEX if bad else pkg.DSV4_OK)
    assert np.array_equal(got[adds == 0], table[adds == 0])          # places that no token lists are left as they were
    tol = 642 * 2.0 ** -23 * bound + (2.0 ** -20 + 2.0 ** -17) * (want - table) + adds * 2.0 ** -24 * np.abs(want) + 1e-37
    err = np.abs(got - want)
    at = adds > 0
    assert np.all(err[at] <= tol[at]), ((err[at] / tol[at]).max(), np.argwhere(at & ~(err <= tol))[:3])
    return got


def both(w):
    return [w, to_fp4(w)]


@pytest.mark.parametrize("heads", [16, 32, 64, 128])
@pytest.mark.parametrize("kind", [0, 1])
def test_heads(heads, kind):
    need_gpu()
    w = synth.make_workload(name="w", seed=heads, heads=heads, req_seq_lens=[700, 33, 1, 260], topk_width=200, window=50,
                            sink=heads == 64)
    check(both(w)[kind], gap=3)


@pytest.mark.parametrize("seqs,K,W", [([1], 1, 1), ([2, 1, 0], 0, 1), ([0, 3], 4, 4), ([127, 128, 129], 0, 300), ([64, 65, 63], 70, 0),
                                      ([513, 512, 511], 384, 128), ([5000], 17, 4000), ([90] * 40, 60, 7)])
@pytest.mark.parametrize("kind", [0, 1])
def test_lengths(seqs, K, W, kind):
    need_gpu()
    w = synth.make_workload(name="w", seed=len(seqs) + K, heads=16, req_seq_lens=seqs, topk_width=K, window=W, sink=False)
    check(both(w)[kind])


@pytest.mark.parametrize("heads", [16, 128])
def test_junk_in_the_lists(heads):
    need_gpu()
    check(junk_workload(heads))
    check(to_fp4(edge_workload(heads, True)))


@pytest.mark.parametrize("kind", [0, 1])
def test_tokens_that_share_rows_are_added_in_order(kind):
    need_gpu()
    w = both(synth.make_workload(name="w", seed=5, heads=32, req_seq_lens=[900, 300, 512], tokens_per_req=3, topk_width=100,
                                 window=64, sink=True))[kind]
    assert len(set(w.req_idx.tolist())) == 3
    first = check(w)
    for _ in range(3):
        assert np.array_equal(run(w, lse_of(w), start_table(w))[0], first)      # the same bits again
    # scattered over the batch, in another order of rows
    rng = np.random.default_rng(6)
    order = rng.permutation(w.num_tokens)
    v = dataclasses.replace(w, q=w.q[order], req_idx=w.req_idx[order], topk_idx=w.topk_idx[order], seq_lens=w.seq_lens[order],
                            topk_lens=None if w.topk_lens is None else w.topk_lens[order])
    check(v)


def test_many_tokens_of_one_row():
    need_gpu()
    w = synth.make_workload(name="w", seed=9, heads=16, req_seq_lens=[700], tokens_per_req=90, topk_width=40, window=30, sink=False)
    check(w)


@pytest.mark.parametrize("rows", [65536, 140000])
def test_tables_of_many_rows(rows):
    need_gpu()
    w = synth.make_workload(name="w", seed=12, heads=16, req_seq_lens=[30, 17, 44], tokens_per_req=2, topk_width=6, window=9, sink=False,
                            page=16)
    table = np.full((rows, w.block_table.shape[1]), -1, np.int32)
    at = np.array([rows - 1, 0, rows // 2])
    table[at] = w.block_table
    check(dataclasses.replace(w, block_table=table, req_idx=at[w.req_idx].astype(np.int32)))


@pytest.mark.parametrize("heads,kind", [(16, 0), (128, 0), (128, 1)])
def test_long_runs_across_tokens(heads, kind):
    need_gpu()
    seqs = np.random.default_rng(heads).integers(700, 1500, 96)          # 9 blocks to a token, 5 to a multiprocessor
    seqs[[3, 50, 51]] = 0, 1, 0
    w = both(synth.make_workload(name="w", seed=13, heads=heads, req_seq_lens=seqs, topk_width=40, window=1300, sink=False))[kind]
    check(w)


def test_hundreds_of_tokens_of_few_rows():
    need_gpu()
    w = synth.make_workload(name="w", seed=10, heads=16, req_seq_lens=[500, 260, 300], tokens_per_req=110, topk_width=12, window=9,
                            sink=False)
    order = np.random.default_rng(1).permutation(w.num_tokens)
    check(dataclasses.replace(w, q=w.q[order], req_idx=w.req_idx[order], topk_idx=w.topk_idx[order], seq_lens=w.seq_lens[order]))


def test_more_tokens_than_threads():
    need_gpu()
    w = synth.make_workload(name="w", seed=11, heads=16, req_seq_lens=np.random.default_rng(2).integers(0, 90, 1900), topk_width=6,
                            window=3, sink=False, page=16)
    check(w)
    check(to_fp4(w))


@pytest.mark.parametrize("entry", [400, 656])
def test_a_cache_past_four_gigabytes(entry):
    need_gpu()
    # a few pages at both ends of a pool of 4.7 GB
    w = synth.make_workload(name="w", seed=18, heads=16, req_seq_lens=[700, 300], topk_width=100, window=64, sink=False)
    w = w if entry == 656 else to_fp4(w)
    lse, table = lse_of(w), start_table(w)
    n, B = len(w.kv_cache), 4_700_000_000 // (64 * entry)
    to = np.where(np.arange(n) % 2, np.arange(n), B - 1 - np.arange(n)).astype(np.int32)
    pool = torch.zeros(B, 64, entry, dtype=torch.uint8, device="cuda")
    pool[torch.from_numpy(to.astype(np.int64)).cuda()] = torch.from_numpy(w.kv_cache).cuda()
    t = np.where(w.block_table >= 0, to[w.block_table], -1).astype(np.int32)
    far, status = run(dataclasses.replace(w, block_table=t), lse, table, kv_cache=pool)
    assert status == pkg.DSV4_OK and np.array_equal(far, run(w, lse, table)[0])


def test_beside_a_decode_and_matrix_products_on_other_streams():
    need_gpu()
    ws = both(synth.make_workload(name="w", seed=19, heads=128, req_seq_lens=[900, 300, 512, 77] * 20, topk_width=200, window=64,
                                  sink=False))
    ds = [synth.to_device(w, "cuda") for w in ws]
    decode = [pkg.sparse_mla_decode, pkg.sparse_mla_decode_fp4]
    lses = [f(**d)[1] for f, d in zip(decode, ds)]
    a = torch.randn(1024, 1024, device="cuda").bfloat16()
    spaces = [pkg.workspace_for_key_weights(w.num_tokens, 128, 200, 64) for w in ws]
    tables = [torch.zeros(len(w.block_table), w.block_table.shape[1] * w.page, device="cuda") for w in ws]

    def weights(i, t):
        args = {n: v for n, v in ds[i].items() if n != "sink"}
        pkg.check(pkg.dsv4_sparse_mla_key_weights(lse=lses[i], weights=t, workspace=spaces[i], **args))
    want = []
    for i in range(2):
        t = tables[i].clone()
        weights(i, t)
        want.append(t)
    outs, product = [f(**d)[0] for f, d in zip(decode, ds)], a @ a
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    got, other = [], []
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                t = torch.zeros_like(tables[i])
                weights(i, t)
                got.append((i, t))
        with torch.cuda.stream(streams[2]):
            other.append([f(**d)[0] for f, d in zip(decode, ds)])
        with torch.cuda.stream(streams[3]):
            other.append(a @ a)
    torch.cuda.synchronize()
    assert all(torch.equal(t, want[i]) for i, t in got)
    assert all(torch.equal(o, product) if torch.is_tensor(o) else all(map(torch.equal, o, outs)) for o in other)
    pkg.check(pkg.dsv4_get_device_status())


def test_bad_pages_rows_and_lengths():
    need_gpu()
    w = synth.make_workload(name="w", seed=5, heads=16, req_seq_lens=[900, 300, 512, 77], topk_width=100, window=64, sink=False)
    t = w.block_table.copy()
    t[0, 1], t[1, 2], t[2, 0] = -1, len(w.kv_cache), 2 ** 31 - 1
    lse = lse_of(w)
    check(dataclasses.replace(w, block_table=t), lse)
    check(dataclasses.replace(w, req_idx=np.array([0, -1, 4, 3], np.int32)), lse)
    s = w.seq_lens.copy()
    s[1], s[2] = -2 ** 31, t.shape[1] * w.page + 40
    check(dataclasses.replace(w, seq_lens=s), lse)


def test_lse_that_is_infinite():
    need_gpu()
    w = synth.make_workload(name="w", seed=7, heads=16, req_seq_lens=[300, 200], topk_width=50, window=20, sink=False)
    lse = lse_of(w)
    lse[0, 3], lse[0, 5], lse[1, :] = -np.inf, np.inf, -np.inf
    got = check(w, lse)
    assert np.array_equal(got[1], start_table(w)[1])


def test_large_logits_and_scales():
    need_gpu()
    w = synth.make_workload(name="w", seed=8, heads=16, req_seq_lens=[300, 200], topk_width=50, window=20, sink=False)
    for s in (0.0, 1e-3, 0.5):
        v = dataclasses.replace(w, softmax_scale=s)
        check(v)
    check(to_fp4(w, spread=3))


def test_entries_that_nobody_lists_may_be_nan():
    need_gpu()
    from fp4_util import unlisted_as_nan
    w = synth.make_workload(name="w", seed=12, heads=64, req_seq_lens=[300, 130, 1], topk_width=50, window=20, sink=False)
    for v in both(w):
        lse = lse_of(v)
        assert np.array_equal(check(unlisted_as_nan(v), lse), check(v, lse))


def test_nan_entries_reach_their_own_place_alone():
    need_gpu()
    for w in both(synth.make_workload(name="w", seed=13, heads=16, req_seq_lens=[300, 130], topk_width=50, window=20, sink=False)):
        lse = lse_of(w)
        clean = run(w, lse, start_table(w))[0]
        cache = w.kv_cache.copy()
        p = int(w.seq_lens[0]) - 3                       # in the window of token 0
        cache[w.block_table[0, p // w.page], p % w.page] = 255
        got = run(dataclasses.replace(w, kv_cache=cache), lse, start_table(w))[0]
        assert np.isnan(got[0, p])
        got[0, p] = clean[0, p]
        assert np.array_equal(got, clean)


def test_wide_rows_of_queries_and_streams():
    need_gpu()
    w = synth.make_workload(name="w", seed=14, heads=32, req_seq_lens=[300, 130, 64], topk_width=50, window=20, sink=False)
    d = synth.to_device(w, "cuda")
    wide = torch.zeros(3, 32 * 576 + 64, dtype=torch.bfloat16, device="cuda")
    wide[:, 64:] = d["q"].reshape(3, -1)
    check(w, q=wide[:, 64:].view(3, 32, 576), stream=torch.cuda.Stream())


def test_what_the_decode_returned_is_spread_over_the_keys():
    need_gpu()
    for w in both(synth.make_workload(name="w", seed=15, heads=64, req_seq_lens=[3000, 2000, 500], topk_width=512, window=128,
                                      sink=False)):
        d = synth.to_device(w, "cuda")
        f = pkg.sparse_mla_decode if w.kv_cache.shape[2] == 656 else pkg.sparse_mla_decode_fp4
        _, lse = f(**d)
        d.pop("sink")
        weights = pkg.sparse_mla_key_weights(lse=lse, **d)
        # each head's weights sum to 1; both kernels' logits are within 642 * 2^-23 * 20 of the same ones
        assert torch.allclose(weights.sum(1).double(), torch.full((3,), 64.0, dtype=torch.float64, device="cuda"), rtol=4e-3)


def test_graph_replays_add_again():
    need_gpu()
    w = synth.make_workload(name="w", seed=16, heads=16, req_seq_lens=[300, 130], tokens_per_req=2, topk_width=50, window=20,
                            sink=False)
    d = synth.to_device(w, "cuda")
    d.pop("sink")
    lse = torch.from_numpy(lse_of(w)).cuda()
    ws = pkg.workspace_for_key_weights(w.num_tokens, 16, 50, 20)
    once = pkg.sparse_mla_key_weights(lse=lse, **d)
    weights = torch.zeros_like(once)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkg.check(pkg.dsv4_sparse_mla_key_weights(lse=lse, weights=weights, workspace=ws, **d))
    assert not bool(weights.any())
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(weights, once)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.allclose(weights, 2 * once, rtol=2.0 ** -22, atol=0)    # four roundings


def test_refusals():
    need_gpu()
    w = synth.make_workload(name="w", seed=17, heads=16, req_seq_lens=[30, 13], topk_width=5, window=2, sink=False)
    d = synth.to_device(w, "cuda")
    d.pop("sink")
    lse = torch.zeros(2, 16, device="cuda")
    table = torch.zeros(2, w.block_table.shape[1] * w.page, device="cuda")
    ws = pkg.workspace_for_key_weights(2, 16, 5, 2)
    f = pkg.dsv4_sparse_mla_key_weights
    assert f(lse=lse, weights=table[:, :-1], workspace=ws, **d) == pkg.DSV4_ERR_INVALID_ARG
    assert f(lse=lse, weights=table, workspace=ws[:-256], **d) == pkg.DSV4_ERR_INVALID_ARG
    assert f(lse=lse, weights=table, workspace=ws, **{**d, "kv_cache": d["kv_cache"][..., :640].contiguous()}) == pkg.DSV4_ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        f(lse=lse[:, :8], weights=table, workspace=ws, **d)
    with pytest.raises(ValueError):
        f(lse=lse, weights=table[:1], workspace=ws, **d)
    with pytest.raises(ValueError):
        f(lse=lse, weights=table, workspace=ws, **{**d, "kv_cache": d["kv_cache"][:, ::2]})
    with pytest.raises(TypeError):
        f(lse=lse.double(), weights=table, workspace=ws, **d)
    assert not bool(table.any())
