"""The 4-bit insert's codes where the normalised key lies within a few fp32 roundings of a border between two codes: the entry
is that of the exact key."""
import numpy as np
import pytest
import torch

import sparse_mla_decode_combine_gb300 as pkg
import synth
from gpu_util import need_gpu
from oracle import fp4
from test_gpu_insert_fp4 import bf16, run_case, table_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("norm_dims", [512, 576])
@pytest.mark.parametrize("spread", [1.0, 30.0])
def test_values_within_a_few_roundings_of_a_border(norm_dims, spread):
    """Every token has the same values at the even dims, and a permutation of the same ones at the odd dims: the root is the
    same, what the sum of squares is rounded to is not.  The weights put the even dims' values within 2^-20 of borders on either
    side; each block's largest value is 4.5, so that its scale is 1."""
    need_gpu()
    rng = np.random.default_rng(norm_dims + int(spread))
    T = 3000
    x = fp4.bf16_to_f64(synth.bf16_bits(rng.standard_normal(576) * np.exp(rng.uniform(0, np.log(spread), 576))))
    x[x == 0] = 1.0
    odd = np.arange(1, norm_dims, 2)
    rows = np.tile(x, (T, 1))
    for t in range(T):
        rows[t, odd] = x[rng.permutation(odd)] * rng.choice([-1.0, 1.0], len(odd))
    root = np.sqrt((x[:norm_dims] ** 2).mean() + 1e-6)
    w = np.zeros(norm_dims)
    target = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], 512) * (1 + rng.uniform(-1, 1, 512) * 2.0 ** -20)
    target[target > 4.9] = 1.75
    target[::32] = 4.5
    w[:512:2] = (target * root / np.abs(x[:512]))[::2]
    w[512:] = 1.0
    w = w.astype(np.float32)
    kv = synth.bf16_bits(rows)
    table = table_of(rng, 8)
    pos, slots = rng.integers(0, 8, T), rng.permutation(T)
    q = np.full((T, 1, 576), 0x3F80, np.uint16)
    want = fp4.insert(q, kv, pos, slots, table, np.zeros((T, 400), np.uint8), None, w, norm_dims, 1e-6)[2]
    cache = torch.zeros((T, 400), dtype=torch.uint8, device="cuda")
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    pkg.check(pkg.dsv4_qk_norm_rope_kv_insert_fp4(bf16(q), bf16(q), bf16(kv), dev(pos), dev(slots), dev(table), cache, None, None,
                                                  dev(w), norm_dims, 1e-6))
    got = cache.cpu().numpy()
    same = np.r_[0:256, 384:400]
    assert np.all(want[:, 384:400] == 127)
    assert np.array_equal(got[:, same], want[:, same]), np.argwhere(got[:, same] != want[:, same])[:4]


def test_many_tokens_are_exact_over_all_dims():
    """As over the latent alone: four million values that are normalised with the rope part."""
    need_gpu()
    run_case(408, T=8000, H=1, norm_dims=576, weights=True, bad=False)
