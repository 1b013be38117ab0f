"""dsv4_sparse_mla_decode_fp4 where logits are -inf: such a key has no weight, a head whose logits are all -inf has no key.

A key's logit is -inf for every head through one infinite rope value that every query meets with a negative one.  The oracle
then decodes the lists without those keys (its own sum of magnitudes would be infinite, and hide every error)."""
import dataclasses

import numpy as np
import pytest
import torch

import sparse_mla_decode_combine_gb300 as pkg
import synth
from fp4_util import compare, run, to_fp4
from gpu_util import need_gpu
from oracle import fp4

pytestmark = pytest.mark.gpu

FEW, MANY, SPLIT = (3, 16), (170, 64), (90, 128)     # units: few and shared, about one a CTA, split between runs


def workload(tokens, heads, keys, dead, sink, low=-200.0):
    """Tokens over the first `keys` positions of their histories, in order; the positions in `dead` have logits of -inf,
    the others' lie around `low` and below."""
    w = to_fp4(synth.make_workload(name=f"{tokens} x {heads}", seed=96, heads=heads, req_seq_lens=[keys] * tokens, topk_width=keys,
                                   window=0, sink=sink))
    cache = w.kv_cache.copy()
    rope = np.zeros((cache.shape[0], w.page, 64))
    rope[..., 1] = 1.0
    for t in range(tokens):
        for p in dead:
            rope[w.block_table[t, p // w.page], p % w.page, 0] = np.inf
    cache[..., 256:384] = synth.bf16_bits(rope).astype("<u2").view(np.uint8).reshape(*cache.shape[:2], 128)
    q = fp4.bf16_to_f64(w.q)
    q[..., :512] *= 0.1
    q[..., 512:] = 0.0
    q[..., 512] = -1.0
    q[..., 513] = (low - 3.0 * np.arange(heads))[None]
    w = dataclasses.replace(w, kv_cache=cache, q=synth.bf16_bits(q), softmax_scale=1.0,
                            topk_idx=np.tile(np.arange(keys, dtype=np.int32), (tokens, 1)), topk_lens=None)
    live = w.topk_idx.copy()
    live[:, list(dead)] = -1
    return w, dataclasses.replace(w, topk_idx=live)


def check(w, live):
    out, lse, st = run(w)
    assert st == pkg.DSV4_OK
    idx = sorted({0, 1, w.num_tokens // 2, w.num_tokens - 1})
    compare(out[idx], lse[idx], fp4.decode(live, idx), w.name)


@pytest.mark.parametrize("sink", [False, True])
@pytest.mark.parametrize("tokens,heads", [FEW, MANY, SPLIT])
@pytest.mark.parametrize("keys", [1, 64, 200])
def test_every_logit_is_minus_infinity(tokens, heads, keys, sink):
    """The same as a token without a key, however its work is split: out = 0, lse = the sink (or -inf)."""
    need_gpu()
    w, _ = workload(tokens, heads, keys, range(keys), sink)
    out, lse, st = run(w)
    want = np.tile(w.sink if sink else np.full(heads, -np.inf, np.float32), (tokens, 1))
    assert st == pkg.DSV4_OK and not out.any() and np.array_equal(lse.cpu().numpy(), want)


@pytest.mark.parametrize("sink", [False, True])
@pytest.mark.parametrize("tokens,heads", [FEW, MANY, SPLIT])
@pytest.mark.parametrize("dead", [[0], range(64), range(130), [0, 64, 128, 199], range(199), [100]])
def test_some_logits_are_minus_infinity(tokens, heads, dead, sink):
    """The first key, all of the first blocks, or keys behind them: the logits that are left lie 200 and more below 0, so no
    reference but one of their own keeps their weights in fp32's range."""
    need_gpu()
    check(*workload(tokens, heads, 200, dead, sink))


@pytest.mark.parametrize("tokens,heads", [FEW, MANY])
def test_the_first_key_is_left_out_and_the_next_is_minus_infinity(tokens, heads):
    """A page out of range at the list's start (no key, flagged), then logits of -inf, then finite ones."""
    need_gpu()
    w, live = workload(tokens, heads, 200, range(64, 100), False)
    table = w.block_table.copy()
    table[:, 0] = -1
    w, live = (dataclasses.replace(x, block_table=table) for x in (w, live))
    out, lse, st = run(w)
    assert st == pkg.DSV4_ERR_BAD_INDEX
    idx = [0, w.num_tokens - 1]
    compare(out[idx], lse[idx], fp4.decode(live, idx))


@pytest.mark.parametrize("tokens,heads", [FEW, MANY, SPLIT, (1, 16)])
def test_a_sink_of_plus_infinity_takes_all_of_the_weight(tokens, heads):
    """lse = +inf and out = 0 for its heads, however the work is split; the other heads are what they are without it."""
    need_gpu()
    keys = 1500 if tokens == 1 else 200
    w, _ = workload(tokens, heads, keys, [], True, low=0.0)
    seqs = w.seq_lens.copy()
    if tokens > 2:
        seqs[2] = 0
    w = dataclasses.replace(w, seq_lens=seqs)
    plain, plain_lse, _ = run(w)
    sink = w.sink.copy()
    sink[::5] = np.inf
    out, lse, st = run(dataclasses.replace(w, sink=sink))
    top = torch.from_numpy(np.isinf(sink)).cuda()
    assert st == pkg.DSV4_OK
    assert not out[:, top].any() and bool(torch.isposinf(lse[:, top]).all())
    assert torch.equal(out[:, ~top], plain[:, ~top]) and torch.equal(lse[:, ~top], plain_lse[:, ~top])
