"""The keys' weights after the verification: with a length of 0 for the tokens that do not stand, the table holds what the tokens that stay
gave their keys, and nothing at the places of those that fell."""
import dataclasses

import numpy as np
import pytest
import torch

import sparse_mla_decode_combine_gb300 as pkg
import synth
from fp4_util import to_fp4
from gpu_util import need_gpu
from oracle import serving
from test_gpu_key_weights import check, lse_of, start_table

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", [0, 1])
def test_weights_of_the_tokens_that_stand(kind):
    need_gpu()
    k, R, V = 3, 5, 400
    w = synth.make_workload(name="w", seed=41 + kind, heads=32, req_seq_lens=[400, 90, 260, 33, 150], tokens_per_req=k + 1, topk_width=50,
                            window=40, sink=False, page=16)
    w = to_fp4(w) if kind else w
    rng = np.random.default_rng(8)
    p = rng.random((R * (k + 1), V)).astype(np.float32)
    tok = rng.integers(0, V, R * k).astype(np.int32)
    start = (np.arange(R + 1) * (k + 1)).astype(np.int32)
    u = np.where(rng.random(len(p)) < 0.6, 0.0, 1.0 - 2.0 ** -24).astype(np.float32)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    _, accepted = pkg.verify_drafts(dev(p), None, dev(tok), dev(start), dev(u), k)
    want = serving.verify(p, None, tok, start, u)[1]
    assert accepted.tolist() == want.tolist() and 0 < want.sum() < R * k
    # row j of a request stands when it comes before the drafts that fell (the first row's token was there before)
    j = torch.arange(k + 1, device="cuda")
    lens = torch.where(j <= accepted[:, None], dev(w.seq_lens).view(R, k + 1), 0).view(-1).contiguous()
    table = start_table(w)
    for r in range(R):                       # (nothing at the places of the drafts)
        table[r, int(w.seq_lens[(k + 1) * r]):] = 0
    got = check(dataclasses.replace(w, seq_lens=lens.cpu().numpy()), lse_of(w), table)
    for r in range(R):
        n = int(w.seq_lens[(k + 1) * r]) + int(want[r])
        assert (got[r, :n] > 0).all() and not got[r, n:].any()
