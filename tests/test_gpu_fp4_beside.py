"""The 4-bit decode beside other kernels that use the tensor cores and tensor memory, on streams of their own: the 8-bit decode and
a library's matrix products."""
import pytest
import torch

import sparse_mla_decode_combine_gb300 as pkg
import synth
from fp4_util import to_fp4
from gpu_util import need_gpu, small

pytestmark = pytest.mark.gpu


def test_three_kinds_of_kernels_at_once():
    need_gpu()
    w8 = [small(3), small(4)]
    w4 = [to_fp4(w) for w in w8] + [to_fp4(synth.make_workload(name="many", seed=106, heads=64, req_seq_lens=[300] * 100, topk_width=100,
                                                               window=50, sink=True))]
    d8, d4 = [synth.to_device(w, "cuda") for w in w8], [synth.to_device(w, "cuda") for w in w4]
    a, b = (torch.randn((1024, 1024), device="cuda").bfloat16() for _ in range(2))
    want8, want4 = [pkg.sparse_mla_decode(**d) for d in d8], [pkg.sparse_mla_decode_fp4(**d) for d in d4]
    want = a @ b
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got8, got4, products = [], [], []
    for _ in range(30):
        with torch.cuda.stream(streams[0]):
            got8.append([pkg.sparse_mla_decode(**d) for d in d8])
        with torch.cuda.stream(streams[1]):
            got4.append([pkg.sparse_mla_decode_fp4(**d) for d in d4])
        with torch.cuda.stream(streams[2]):
            products.append(a @ b)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for g in got4 for p, q in zip(g, want4) for x, y in zip(p, q))
    assert all(torch.equal(x, y) for g in got8 for p, q in zip(g, want8) for x, y in zip(p, q))
    assert all(torch.equal(p, want) for p in products)
    assert pkg.dsv4_get_device_status() == pkg.DSV4_OK
