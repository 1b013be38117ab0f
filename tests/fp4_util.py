"""Workloads over a cache of 4-bit entries, and the decode's tolerances, shared by the GPU tests."""
from __future__ import annotations

import dataclasses

import numpy as np
import torch

import sparse_mla_decode_combine_gb300 as pkg
import synth
from oracle import fp4


def to_fp4(w: synth.Workload, seed: int = 5, spread: int = 0) -> synth.Workload:
    """The workload with its cache replaced by 4-bit entries: N(0, 1) latents, each block of 32 scaled by a random
    power of two up to 2^+-spread."""
    rng = np.random.default_rng(seed)
    blocks, page, _ = w.kv_cache.shape
    n = min(blocks * page, 6000)
    x = rng.standard_normal((n, 16, 32)) * np.ldexp(1.0, rng.integers(-spread, spread + 1, (n, 16, 1)))
    rows = fp4.pack(x.reshape(n, 512), synth.bf16_bits(rng.standard_normal((n, 64))))
    rows = rows[rng.integers(0, n, blocks * page)] if n < blocks * page else rows
    return dataclasses.replace(w, kv_cache=rows.reshape(blocks, page, fp4.ENTRY_BYTES))


def unlisted_as_nan(w: synth.Workload) -> synth.Workload:
    """Every entry that no token lists becomes NaN (scale bytes 255, NaN rope)."""
    import oracle
    lists, lens = oracle.combine(w.topk_idx, w.topk_lens, w.seq_lens, w.window, w.topk_idx.shape[1] + w.window)
    used = np.zeros(w.kv_cache.shape[:2], bool)
    for t in range(w.num_tokens):
        row = t if w.req_idx is None else int(w.req_idx[t])
        p = lists[t, :lens[t]]
        used[w.block_table[row, p // w.page], p % w.page] = True
    cache = w.kv_cache.copy()
    cache[~used] = 255
    return dataclasses.replace(w, kv_cache=cache)


def run(w: synth.Workload, stream=None, **over):
    """The decode on the GPU, with guards around its outputs and a workspace of stale bytes -> (out, lse, status)."""
    d = {**synth.to_device(w, "cuda"), **over}
    T, H, pad = w.num_tokens, w.num_heads, 64
    out_full = torch.full((T * H * 512 + 2 * pad,), -7.0, dtype=torch.bfloat16, device="cuda")
    lse_full = torch.full((T * H + 2 * pad,), -7.0, dtype=torch.float32, device="cuda")
    ws = pkg.workspace_for_fp4(T, H, w.topk_width, w.window)
    ws.fill_(0xA5)
    out, lse = out_full[pad:-pad].view(T, H, 512), lse_full[pad:-pad].view(T, H)
    torch.cuda.synchronize()
    pkg.dsv4_get_device_status()
    pkg.check(pkg.dsv4_sparse_mla_decode_fp4(out=out, lse=lse, workspace=ws, stream=stream, **d), "decode")
    torch.cuda.synchronize()
    status = pkg.dsv4_get_device_status()
    for full in (out_full, lse_full):
        assert bool((full[:pad] == -7).all()) and bool((full[-pad:] == -7).all()), "write outside an output"
    return out, lse, status


def compare(out, lse, ref, what=""):
    """Against oracle.fp4.decode.  Queries and dequantised keys are exact in BF16, so what rounds is
      a logit:     an fp32 sum of 576 exact products, at most 640 roundings (the tile's order included) of the sum of
                   magnitudes `dot`, each 2^-23 at most (the tensor core may truncate): ds = 640 * 2^-23 * dot;
      a weight:    e^ds, then the exponential and the running maximum's rescaling, 2^-20 together, then BF16: half a
                   step, 2^-8 of the value;
      the output:  the fp32 sum over the keys, 2^-12 of the sum of magnitudes `mag` (8192 + window terms at 2^-25 on
                   average; the bound of the sizes here), and one rounding to BF16, 2^-8 of the value;
      the lse:     ds, the fp32 sum of the weights and the logarithm, 2^-18 together, and fp32's 2^-23 of the value."""
    r_out, r_lse, mag, dot, _ = ref
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    ds = 640 * 2.0 ** -23 * dot
    inf = np.isneginf(r_lse)
    assert np.array_equal(np.isneginf(l), inf), what
    err_l = np.abs(np.where(inf, 0, l) - np.where(inf, 0, r_lse))
    tol_l = ds + 2.0 ** -18 + 2.0 ** -23 * np.abs(np.where(inf, 0, r_lse))
    assert np.all(err_l <= tol_l), (what, "lse", (err_l / tol_l).max())
    tol = (2.0 ** -8 + 2.0 ** -20 + 2.0 ** -12 + 2 * ds[..., None]) * mag + 2.0 ** -8 * np.abs(r_out) + 1e-38
    err = np.abs(o - r_out)
    assert np.all(err <= tol), (what, "out", (err / tol).max(), np.argwhere(~(err <= tol))[:3])
    return (err / tol).max(), (err_l / tol_l).max()
