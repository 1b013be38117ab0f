"""The operators between two decode steps as a serving loop runs them: decode of the drafted tokens, the keys' weights,
verification, eviction, and a decode over what is left; all captured into one graph, and replayed."""
import dataclasses

import numpy as np
import pytest
import torch

import oracle
import sparse_mla_decode_combine_gb300 as pkg
import synth
from fp4_util import to_fp4
from gpu_util import need_gpu
from oracle import fp4, serving

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", [0, 1])
def test_loop(kind):
    need_gpu()
    w = synth.make_workload(name="loop", seed=31 + kind, heads=16, req_seq_lens=[400, 150, 260], tokens_per_req=3, topk_width=80,
                            window=40, sink=True, page=16)
    w = to_fp4(w) if kind else w
    R, T, V, k = 3, 9, 5000, 2
    rng = np.random.default_rng(7)
    d = synth.to_device(w, "cuda")
    decode = pkg.sparse_mla_decode_fp4 if kind else pkg.sparse_mla_decode
    oracle_decode = (lambda v: fp4.decode(v)[:2]) if kind else (lambda v: oracle.sparse_mla_decode(v)[:2])
    z = 2 * rng.standard_normal((T, V))
    p = torch.softmax(torch.from_numpy(z), 1).float().cuda()
    rows = [0, 1, 3, 4, 6, 7]
    q = torch.softmax(torch.from_numpy(z[rows] + 0.5 * rng.standard_normal((6, V))), 1).float().cuda()
    tok = q.argmax(1).int()
    start = torch.arange(0, T + 1, k + 1, dtype=torch.int32, device="cuda")
    uniform = torch.from_numpy(rng.random(T).astype(np.float32)).cuda()
    lens = torch.tensor([400, 150, 260], dtype=torch.int32, device="cuda")
    refs = torch.zeros(len(w.kv_cache), dtype=torch.int32, device="cuda")
    refs[d["block_table"][d["block_table"] >= 0].long()] = 1
    pool = d["kv_cache"][None]
    table = torch.zeros(R, w.block_table.shape[1] * w.page, device="cuda")
    budget, first, recent = 120, 4, 48
    none = torch.empty(R, 0, dtype=torch.int32, device="cuda")
    got = {}

    def step():
        out, lse = decode(**d)
        weights = pkg.sparse_mla_key_weights(lse=lse, **{n: v for n, v in d.items() if n != "sink"}, weights=table)
        tokens, accepted, new = pkg.verify_drafts(p, q, tok, start, uniform, k, seq_lens=lens)
        bt, n, rc, left = pkg.cache_evict(pool, d["block_table"], new, refs, weights, budget, None, first, recent)
        after = decode(d["q"][::3].contiguous(), pool[0], bt, None, none, None, n, 200, None, 0.04)
        got.update(lse=lse, weights=weights, tokens=tokens, accepted=accepted, new=new, bt=bt, n=n, rc=rc, left=left, out=after[0],
                   after=after[1])

    cache = pool.clone()
    step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        step()
    for _ in range(2):
        pool.copy_(cache)
        table.zero_()
        graph.replay()
        torch.cuda.synchronize()
        pkg.check(pkg.dsv4_get_device_status())
        h = {n: v.cpu().numpy() for n, v in got.items() if n != "out"}
        want_w, _, _, _ = serving.key_weights(w, h["lse"], np.zeros(table.shape))
        assert np.allclose(h["weights"], want_w, rtol=4e-3, atol=1e-6)
        out, acc, seq, may, _ = serving.verify(p.cpu().numpy(), q.cpu().numpy(), tok.cpu().numpy(), start.cpu().numpy(),
                                               uniform.cpu().numpy(), seq=np.array([400, 150, 260], np.int32))
        assert np.array_equal(h["accepted"], acc) and np.array_equal(h["new"], seq)
        assert all(int(h["tokens"][b, acc[b]]) in may[b] for b in range(R))
        c, bt, n, rc, left, bad = serving.evict(cache.cpu().numpy(), w.block_table, seq, refs.cpu().numpy(), h["weights"], budget,
                                                budget, first, recent)
        assert bad == 0 and np.array_equal(pool.cpu().numpy(), c)
        for name, ref in (("bt", bt), ("n", n), ("rc", rc), ("left", left)):
            assert np.array_equal(h[name], ref), name
        v = dataclasses.replace(w, q=w.q[::3], kv_cache=c[0], block_table=bt, req_idx=None, topk_idx=np.zeros((R, 0), np.int32),
                                topk_lens=None, seq_lens=n, window=200, sink=None, softmax_scale=0.04)
        want, wlse = oracle_decode(v)
        assert np.abs(got["out"].double().cpu().numpy() - want).max() <= 2e-2 and np.abs(h["after"] - wlse).max() <= 1e-3
