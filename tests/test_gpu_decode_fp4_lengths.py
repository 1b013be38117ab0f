"""dsv4_sparse_mla_decode_fp4 at the ends of the ranges of its lengths."""
import dataclasses

import numpy as np
import pytest
import torch

import sparse_mla_decode_combine_gb300 as pkg
import synth
from fp4_util import run, to_fp4
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,topk", [(2, 40), (2, 1400), (90, 40)])
def test_lengths_below_zero_are_empty(tokens, topk):
    """Down to the type's lowest value, in lists made by the decode and by the list kernel: no key, whatever the row names."""
    need_gpu()
    w = to_fp4(synth.make_workload(name="negative", seed=97, heads=64, req_seq_lens=[200] * tokens, topk_width=topk, window=16,
                                   sink=True))
    w = dataclasses.replace(w, seq_lens=np.resize(np.array([-2 ** 31, -1], np.int32), tokens))
    out, lse, st = run(w)
    assert st == pkg.DSV4_OK and not out.any() and np.array_equal(lse.cpu().numpy(), np.tile(w.sink, (tokens, 1)))
