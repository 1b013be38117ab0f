"""dsv4_sparse_mla_decode_fp4 over entries that are not finite: a product past BF16's range is an infinity in its own dim, scale
byte 255 makes its token NaN, and tokens beside it in the same CTA's run are what they are alone."""
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


def two_keys(tokens, heads):
    """Tokens over keys 0 and 1; queries are zero but for -1 in dim 96 and 1 in dim 200."""
    w = to_fp4(synth.make_workload(name="two keys", seed=101, heads=heads, req_seq_lens=[2] * tokens, topk_width=0, window=2,
                                   sink=False))
    cache = w.kv_cache.copy()
    cache[:, :, 256:384] = 0
    q = np.zeros(w.q.shape)
    q[..., 96], q[..., 200] = -1.0, 1.0
    return dataclasses.replace(w, kv_cache=cache, q=synth.bf16_bits(q), softmax_scale=1.0), cache


def set_code(entry, dim, code):
    b, shift = dim // 2, 4 * (dim % 2)
    entry[b] = (entry[b] & (0xF0 >> shift)) | (code << shift)


@pytest.mark.parametrize("tokens,heads", [(2, 16), (90, 128), (700, 16)])
@pytest.mark.parametrize("inf_key", [0, 1])
def test_a_product_past_bf16_is_an_infinity_in_its_dim(tokens, heads, inf_key):
    """4 * 2^126 is one, 3 * 2^126 is finite.  The key's logit is -inf, so the other key has all of the weight: its latent,
    exactly, in every dim but that of the infinity, which 0 times it makes NaN."""
    need_gpu()
    w, cache = two_keys(tokens, heads)
    want = []
    for t in range(tokens):
        page = cache[w.block_table[t, 0]]
        e, other = page[inf_key], page[1 - inf_key]
        set_code(other, 96, 0)
        e[48:64], e[384 + 3] = 0, 253                  # dims 96 .. 127 under 2^126
        set_code(e, 96, 6)
        set_code(e, 100, 5)
        want.append(fp4.dequant(other)[0])
    out, lse, st = run(w)
    assert st == pkg.DSV4_OK
    o, l, want = out.double().cpu().numpy(), lse.double().cpu().numpy(), np.stack(want)
    dims = np.r_[0:96, 97:512]
    assert np.array_equal(o[:, :, dims], np.repeat(want[:, None, dims], heads, 1)) and np.isnan(o[:, :, 96]).all()
    assert np.all(np.abs(l - want[:, 200, None]) <= 2.0 ** -20)      # (one product; what the logarithm's unit rounds away)


@pytest.mark.parametrize("tokens,heads", [(2, 16), (90, 128), (700, 16)])
def test_the_nan_scale_stays_in_its_token(tokens, heads):
    need_gpu()
    w, cache = two_keys(tokens, heads)
    bad = np.arange(tokens) % 3 == 1
    alone, alone_lse, _ = run(w)
    for t in np.flatnonzero(bad):
        cache[w.block_table[t, 0], t % 2, 384 + t % 16] = 255
    out, lse, st = run(w)
    assert st == pkg.DSV4_OK
    good = torch.from_numpy(~bad).cuda()
    assert bool(torch.isfinite(alone).all())
    assert torch.equal(out[good], alone[good]) and torch.equal(lse[good], alone_lse[good])
    assert bool(torch.isnan(out[~good]).all()) and bool(torch.isnan(lse[~good]).all())


@pytest.mark.parametrize("tokens,heads", [(2, 64), (90, 128)])
@pytest.mark.parametrize("step", [0.03, 0.5])
def test_latents_up_to_2_to_the_64_beside_rising_logits(tokens, heads, step):
    """The largest magnitudes for which the sums are promised to stay finite, with logits that rise over the list to just below
    the range that is left above the first one's (0.03 a key), or past it many times (0.5)."""
    need_gpu()
    keys = 900
    w = to_fp4(synth.make_workload(name="large", seed=102, heads=heads, req_seq_lens=[keys] * tokens, topk_width=0, window=keys,
                                   sink=False))
    cache = w.kv_cache.copy()
    cache[..., 384:] = 127 + 61                            # 6 * 2^61 < 2^64
    rope = np.zeros((*cache.shape[:2], 64))
    for t in range(tokens):
        for i in range(-(-keys // w.page)):
            rope[w.block_table[t, i], :, 0] = step * (64 * i + np.arange(64))
    cache[..., 256:384] = synth.bf16_bits(rope).astype("<u2").view(np.uint8).reshape(*cache.shape[:2], 128)
    q = np.zeros(w.q.shape)
    q[..., 512] = 1.0
    w = dataclasses.replace(w, kv_cache=cache, q=synth.bf16_bits(q), softmax_scale=1.0)
    out, lse, st = run(w)
    assert st == pkg.DSV4_OK
    idx = [0, tokens // 2, tokens - 1]
    compare(out[idx], lse[idx], fp4.decode(w, idx), w.name)
