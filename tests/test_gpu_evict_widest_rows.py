"""Eviction on the GPU with rows of nearly 2^31 entries and tables of 2^31 - 1 weights: positions and tiles past the last one do not
wrap around."""
import pytest
import torch

import sparse_mla_decode_combine_gb300 as pkg
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

PAGE, PAGES, WIDTH = 2047, 1 << 20, 2 ** 31 - 1
MOST = PAGE * PAGES


def evict(table, n, refs, weights, out, budget, limit, first, recent):
    i32 = dict(dtype=torch.int32, device="cuda")
    cache = torch.zeros(1, 1, PAGE, 16, dtype=torch.uint8, device="cuda")
    lens, refs = torch.tensor([n], **i32), torch.tensor([refs], **i32)
    table_out, lens_out, refs_out = torch.empty_like(table), torch.empty_like(lens), torch.empty_like(refs)
    ws = pkg.workspace_for_cache_evict(1, PAGES, 1, 1, PAGE, 16, budget)
    torch.cuda.synchronize()
    pkg.dsv4_get_device_status()
    pkg.check(pkg.dsv4_cache_evict(cache, table, lens, refs, weights, budget, limit, first, recent, table_out, lens_out, refs_out, out, ws))
    torch.cuda.synchronize()
    return table_out, int(lens_out), int(refs_out), pkg.dsv4_get_device_status()


@pytest.fixture(scope="module")
def weights():
    need_gpu()
    torch.manual_seed(1)
    yield torch.rand(1, WIDTH, device="cuda") + 0.5
    torch.cuda.empty_cache()


def test_a_row_that_is_not_cut(weights):
    # more than a round of weights to a CTA, the second of which ends past 2^31
    n, table = MOST - 5, torch.zeros(1, PAGES, dtype=torch.int32, device="cuda")
    out = torch.full_like(weights, 7.0)
    got = evict(table, n, PAGES, weights, out, 1_500_000_000, MOST, 1, 1)
    assert torch.equal(got[0], table) and got[1:] == (n, PAGES, pkg.DSV4_OK)
    assert torch.equal(out[:, :n], weights[:, :n]) and not bool(out[:, n:].any())


def test_a_row_that_loses_a_hundred_entries(weights):
    # (on pages out of range, which are flagged: the weights alone move)
    gone, first = 100, 1_000_000_001
    table = torch.full((1, PAGES), -1, dtype=torch.int32, device="cuda")
    out = torch.full_like(weights, 7.0)
    got = evict(table, MOST, 0, weights, out, MOST - gone, MOST - gone, first, MOST - gone - first)
    assert torch.equal(got[0], table) and got[1:] == (MOST - gone, 0, pkg.DSV4_ERR_BAD_INDEX)
    assert torch.equal(out[:, :first], weights[:, :first]) and not bool(out[:, MOST - gone:].any())
    assert torch.equal(out[:, first:MOST - gone], weights[:, first + gone:MOST])
    kept = weights[:, first + gone:MOST].clone()
    evict(table, MOST, 0, weights, weights, MOST - gone, MOST - gone, first, MOST - gone - first)
    assert torch.equal(weights[:, first:MOST - gone], kept) and not bool(weights[:, MOST - gone:].any())
