"""The allocating wrappers of the 4-bit and page operators on a stream given as an object or as a bare handle: what they
allocate belongs to the stream that the kernels run on."""
import pytest
import torch

import sparse_mla_decode_combine_gb300 as pkg
import synth
from fp4_util import compare, to_fp4
from gpu_util import need_gpu, small
from oracle import fp4

pytestmark = pytest.mark.gpu


class Handle:
    """Another library's stream object: only its handle is known."""

    def __init__(self, cuda_stream):
        self.cuda_stream = cuda_stream


def test_allocations_belong_to_the_stream_of_the_call():
    need_gpu()
    other = torch.cuda.Stream()
    for stream, want in ((None, torch.cuda.current_stream().cuda_stream), (other, other.cuda_stream),
                         (other.cuda_stream, other.cuda_stream), (Handle(other.cuda_stream), other.cuda_stream),
                         (0, 0), (Handle(0), 0), (torch.cuda.default_stream(), 0)):
        with torch.cuda.stream(torch.cuda.Stream()) if stream is not None else torch.cuda.stream(None):
            with pkg._allocating_on(stream):
                assert torch.cuda.current_stream().cuda_stream == want, stream


@pytest.mark.parametrize("how", ["zero", "handle", "object"])
def test_wrappers_on_a_stream_given_by_its_handle(how):
    need_gpu()
    side = torch.cuda.Stream()
    stream = {"zero": 0, "handle": side.cuda_stream, "object": Handle(side.cuda_stream)}[how]
    w = to_fp4(small(1))
    d = synth.to_device(w, "cuda")
    torch.cuda.synchronize()
    out, lse = pkg.sparse_mla_decode_fp4(**d, stream=stream)
    cache = torch.zeros((1, 8, 4, 16), dtype=torch.uint8, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    state = i32(5, 6).view(1, 2), i32(7), i32(0, 0, 0, 0, 0, 1, 1, 0)
    parent = i32(0, 0)
    torch.cuda.synchronize()
    table, lens, refs = pkg.cache_fork_rows(cache, *state, parent, stream=stream)
    table, refs, page_map, live = pkg.cache_compact(cache, table, lens, refs, stream=stream)
    torch.cuda.synchronize()
    compare(out, lse, fp4.decode(w))
    # page 5 (full) shared, page 6 kept by the first child, page 0 taken by the second; then 5 and 6 move to 1 and 2
    assert table.tolist() == [[1, 2], [1, 0]] and refs.tolist() == [1, 2, 1, 0, 0, 0, 0, 0] and live.item() == 3
    assert page_map.tolist() == [0, -1, -1, -1, -1, 1, 2, -1]
