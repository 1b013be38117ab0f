"""dsv4_sparse_mla_decode_fp4: keys of very small weight where the heaviest key's latent is zero, so that they are the output.

Weights are fp32 numbers: one of 2^-120 is kept to its own precision, however the references rose on the way to it."""
import dataclasses

import numpy as np
import pytest

import sparse_mla_decode_combine_gb300 as pkg
import synth
from fp4_util import run, to_fp4
from gpu_util import need_gpu
from oracle import fp4

pytestmark = pytest.mark.gpu


def check(tokens, heads, keys, logits):
    """Logits (in log2 units, [keys], exact in BF16 steps of 1/4 up to 2^8) through one rope dim; key i has the latent 1 in dims
    32 (i % 16) .. and 0 elsewhere, but for the heaviest key, which has none.  Expected: each block's keys' share of the weight."""
    need_gpu()
    logits = np.asarray(logits, np.float64)
    w = to_fp4(synth.make_workload(name="small", seed=105, heads=heads, req_seq_lens=[keys] * tokens, topk_width=0, window=keys,
                                   sink=False))
    cache = np.zeros_like(w.kv_cache)
    cache[..., 384:] = 127
    rope = np.zeros((*cache.shape[:2], 64))
    for t in range(tokens):
        for i in range(keys):
            b, o = w.block_table[t, i // w.page], i % w.page
            if i != logits.argmax():
                cache[b, o, 16 * (i % 16):16 * (i % 16) + 16] = 0x22
            rope[b, o, 0] = logits[i]
    cache[..., 256:384] = synth.bf16_bits(rope).astype("<u2").view(np.uint8).reshape(*cache.shape[:2], 128)
    q = np.zeros(w.q.shape)
    q[..., 512] = 1.0
    w = dataclasses.replace(w, kv_cache=cache, q=synth.bf16_bits(q), softmax_scale=float(np.float32(np.log(2))))
    out, lse, st = run(w)
    assert st == pkg.DSV4_OK
    held = fp4.bf16_to_f64(synth.bf16_bits(logits))
    wt = np.exp2(held - held.max())
    want = np.array([wt[(np.arange(keys) % 16 == b) & (np.arange(keys) != logits.argmax())].sum() for b in range(16)]) / wt.sum()
    want[want < 2.0 ** -121] = 0                                       # (fp32 may flush what BF16 or fp32 cannot hold in full)
    got = out.double().cpu().numpy().reshape(tokens, heads, 16, 32)
    # the scale's rounding times a logit of 256 at most (2^-24 * 256 ln 2 * 2), the exponentials' 2^-20, BF16's weight and output
    tol = (2.0 ** -8 + 2.0 ** -8 + 2.0 ** -14) * want[:, None]
    bad = np.abs(got - want[:, None]) > tol
    bad[..., want == 0, :] = np.abs(got[..., want == 0, :]) > 2.0 ** -120
    assert not bad.any(), np.unique(np.argwhere(bad)[:, 2])


FORMS = [(1, 16, 1024), (90, 64, 256), (90, 128, 512), (300, 64, 128)]


@pytest.mark.parametrize("tokens,heads,keys", FORMS)
@pytest.mark.parametrize("rise", [45, 80, 120, 160, 200])
def test_a_reference_that_rises_far_at_the_end(tokens, heads, keys, rise):
    """Keys just below the range above the first one (2^39), then one that is `rise` above the first."""
    logits = np.zeros(keys)
    logits[1:keys // 2] = 39.0 - np.arange(keys // 2 - 1) % 17
    logits[keys // 2:] = -60.0
    logits[keys - 7] = rise
    check(tokens, heads, keys, logits)


@pytest.mark.parametrize("tokens,heads,keys", FORMS)
@pytest.mark.parametrize("step", [2.0, 0.5, 30.0])
def test_rising_and_falling_logits(tokens, heads, keys, step):
    for sign in (1, -1):
        check(tokens, heads, keys, np.clip(sign * step * (np.arange(keys) - keys // 2), -200, 200))


@pytest.mark.parametrize("tokens,heads,keys", FORMS)
@pytest.mark.parametrize("seed", range(4))
def test_logits_all_over_the_range(tokens, heads, keys, seed):
    rng = np.random.default_rng(seed)
    check(tokens, heads, keys, np.round(rng.uniform(-120, 120, keys)))
