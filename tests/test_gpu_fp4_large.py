"""The 4-bit decode and insert on batches whose arrays pass 2^31 elements, and on the longest window."""
import numpy as np
import pytest
import torch

import sparse_mla_decode_combine_gb300 as pkg
import synth
from fp4_util import compare, to_fp4
from gpu_util import need_gpu
from oracle import fp4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,heads", [(30001, 128), (70003, 16)])
def test_decode_of_a_large_batch(tokens, heads):
    """Tokens share eight rows of the table; queries, outputs and lse of the first and the last ones against the oracle."""
    need_gpu()
    w = to_fp4(synth.make_workload(name="large", seed=103, heads=heads, req_seq_lens=[150, 90, 64, 1, 65, 0, 129, 200], topk_width=60,
                                   window=16, sink=True))
    d = synth.to_device(w, "cuda")
    g = torch.Generator(device="cuda").manual_seed(tokens)
    rows = torch.randint(0, 8, (tokens,), generator=g, device="cuda")
    d["q"] = torch.empty((tokens, heads, 576), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    for k in ("topk_idx", "seq_lens"):
        d[k] = d[k][rows].contiguous()
    d["req_idx"] = rows.int()
    out, lse = pkg.sparse_mla_decode_fp4(**d)
    torch.cuda.synchronize()
    assert pkg.dsv4_get_device_status() == pkg.DSV4_OK
    idx = [0, 1, 2, tokens // 2, tokens - 3, tokens - 2, tokens - 1]
    part = synth.Workload(**{**w.__dict__, "q": d["q"][idx].view(torch.int16).cpu().numpy().view(np.uint16),
                             "req_idx": rows[idx].int().cpu().numpy(), "topk_idx": d["topk_idx"][idx].cpu().numpy(),
                             "seq_lens": d["seq_lens"][idx].cpu().numpy()})
    compare(out[idx], lse[idx], fp4.decode(part))
    # every token of a row without a key is empty, and no other
    empty = rows == 5
    assert not out[empty].any() and torch.equal(lse[empty], d["sink"].expand(int(empty.sum()), heads))
    assert bool(torch.isfinite(lse).all()) and bool(torch.isfinite(out[::97]).all())


@pytest.mark.parametrize("heads", [16, 128])
def test_decode_of_the_longest_window(heads):
    """2^24 keys of one token, positions over a table whose rows name forty pages again and again; queries of zero: the lse is
    ln 2^24, and the output the mean of the pages' latents as often as the table names them."""
    need_gpu()
    n, page = 1 << 24, 64
    w = to_fp4(synth.make_workload(name="longest", seed=104, heads=heads, req_seq_lens=[40 * page], topk_width=0, window=0, sink=False))
    table = np.random.default_rng(1).integers(0, 40, (1, n // page)).astype(np.int32)
    d = synth.to_device(w, "cuda")
    d.update(q=torch.zeros_like(d["q"]), block_table=torch.from_numpy(table).cuda(), window=n,
             seq_lens=torch.tensor([n], dtype=torch.int32, device="cuda"))
    out, lse = pkg.sparse_mla_decode_fp4(**d)
    l = lse.double().cpu().numpy()
    assert np.all(np.abs(l - np.log(n)) <= 2.0 ** -20)                    # (one rounding of 16.6, and the logarithm's)
    latent = fp4.dequant(w.kv_cache).reshape(40, page, 576)[:, :, :512].sum(1)
    share = np.bincount(table[0], minlength=40) / n
    mean, mag = share @ latent, share @ np.abs(fp4.dequant(w.kv_cache).reshape(40, page, 576)[:, :, :512]).sum(1)
    # weights of 1, exact; a part sums 2^24 / 152 keys in 6900 steps of 16, each off by 2^-23 of a partial sum that is half the
    # whole on average, if the tensor core truncates: 6900 * 2^-24 < 2^-11 of the sum of magnitudes; the output's rounding
    assert np.all(np.abs(out.double().cpu().numpy()[0] - mean) <= 2.0 ** -8 * np.abs(mean) + 2.0 ** -11 * mag)
    assert pkg.dsv4_get_device_status() == pkg.DSV4_OK


def test_insert_past_32_bit_offsets():
    """Queries of more than 2^31 elements in place and slots past 2^32 bytes: the last tokens are what they are in a small call."""
    need_gpu()
    T, H, n = 30001, 128, 40
    g = torch.Generator(device="cuda").manual_seed(5)
    q = torch.empty((T, H, 576), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    kv = torch.empty((T, 576), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    slots = 11_000_000
    cache = torch.zeros((slots, 400), dtype=torch.uint8, device="cuda")
    pos = torch.arange(T, device="cuda") % 64
    where = slots - 1 - torch.arange(T, device="cuda")
    cs = torch.randn((64, 64), generator=g, device="cuda")
    small = torch.zeros((n, 400), dtype=torch.uint8, device="cuda")
    want, wk, k = torch.empty((n, H, 576), dtype=torch.bfloat16, device="cuda"), torch.empty_like(kv[:n]), torch.empty_like(kv)
    pkg.check(pkg.dsv4_qk_norm_rope_kv_insert_fp4(q[-n:], want, kv[-n:], pos[-n:], torch.arange(n, device="cuda"), cs, small, wk))
    pkg.check(pkg.dsv4_qk_norm_rope_kv_insert_fp4(q, q, kv, pos, where, cs, cache, k))
    assert torch.equal(q[-n:], want) and torch.equal(k[-n:], wk)
    assert torch.equal(cache[slots - T:slots - T + n].flip(0), small) and not cache[:slots - T].any()
    assert pkg.dsv4_get_device_status() == pkg.DSV4_OK
