"""Key weights on the GPU: a head whose lse is -inf gives nothing, whatever its logits are."""
import dataclasses

import numpy as np
import pytest

import synth
from fp4_util import to_fp4
from gpu_util import need_gpu
from test_gpu_key_weights import check, lse_of, run, start_table

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("heads", [16, 32, 64, 128])
def test_masked_heads_with_any_queries(heads, kind):
    need_gpu()
    w = synth.make_workload(name="w", seed=heads + kind, heads=heads, req_seq_lens=[500, 300, 200, 40], tokens_per_req=2, topk_width=60,
                            window=150, sink=False)
    w = to_fp4(w) if kind else w
    lse = lse_of(w)
    masked = np.random.default_rng(heads).random(lse.shape) < 0.3
    masked[2], masked[3] = False, True       # a token without a masked head, and one of nothing else
    lse[masked] = -np.inf
    q, clean = w.q.copy(), w.q.copy()
    bits = np.array([0x7FC0, 0xFF80, 0x7F80, 0x7F7F, 0xFF7F], np.uint16)     # NaN, the infinities and the largest values
    q[masked] = bits[np.arange(int(masked.sum())) % 5][:, None]
    clean[masked] = 0
    got, _ = run(dataclasses.replace(w, q=q), lse, start_table(w))
    assert np.array_equal(got, check(dataclasses.replace(w, q=clean), lse))
