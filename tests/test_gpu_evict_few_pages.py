"""Eviction on the GPU where there are fewer free pages than shared ones to replace: rows that would need more stay as they were, in every
form of the plan (one cluster's, one CTA's with the selection) and of the selection."""
import numpy as np
import pytest

from gpu_util import need_gpu
from oracle import serving
from test_gpu_evict import check, pool

pytestmark = pytest.mark.gpu


def scarce(seed, lens, free, spare=300, **kw):
    """A pool of which all pages but `free` are held, by its rows or by others that the table does not show."""
    cache, table, lens, refs, w = pool(seed, lens, spare=spare, **kw)
    empty = np.random.default_rng(seed + 1).permutation(np.flatnonzero(refs == 0))
    assert len(empty) >= free
    refs[empty[free:]] = 1 + empty[free:] % 3
    return cache, table, lens, refs, w


def wanted(args, budget, first, recent):
    """How many pages the rows take where there are enough."""
    _, _, _, refs, _, bad = serving.evict(*args, budget, budget, first, recent)
    assert bad == 0
    return int(np.sum((args[3] == 0) & (refs > 0)))


# pages of 4 entries whose first six are shared by two rows each; a budget of 9: up to three pages of a row are written, shared ones
LENS = [30, 30, 25, 31, 24, 24, 40, 9, 40, 40]


@pytest.mark.parametrize("rows", [10, 8, 6, 2])
@pytest.mark.parametrize("in_place", [False, True])
def test_rows_stay_for_want_of_pages(rows, in_place):
    need_gpu()
    need = wanted(scarce(2, LENS[:rows], 100, shared=6), 9, 1, 1)
    assert need >= 2 * (rows - 2)
    for free in range(need + 1):
        want = check(*scarce(2, LENS[:rows], free, shared=6), 9, None, 1, 1, in_place)
        assert (want[5] > 0) == (free < need), (free, want[5])


@pytest.mark.parametrize("in_place", [False, True])
def test_the_last_row_alone_has_no_page(in_place):
    need_gpu()
    need = wanted(scarce(3, [40] * 12, 100, shared=8), 13, 2, 3)
    want = check(*scarce(3, [40] * 12, need - 1, shared=8), 13, None, 2, 3, in_place)
    assert want[5] == 1 and want[2][-1] == 40 and (want[2][:-1] == 13).all()


@pytest.mark.parametrize("rows", [3, 12])
@pytest.mark.parametrize("n,budget", [(700, 300), (3001, 1001), (9000, 2000)])
@pytest.mark.parametrize("in_place", [False, True])
def test_longer_rows(n, budget, rows, in_place):
    need_gpu()
    # the three selections: by counting with 1 and 4 keys to a thread, and the radix select
    lens, kw = [n - 13 * i for i in range(rows)], dict(page=16, entry=48, shared=40, spare=2000)
    need = wanted(scarce(5, lens, 2000, **kw), budget, 4, 50)
    for free in (0, need // 2, need - 1, need):
        want = check(*scarce(5, lens, free, **kw), budget, None, 4, 50, in_place)
        assert (want[5] > 0) == (free < need), free


@pytest.mark.parametrize("in_place", [False, True])
def test_rows_that_stay_are_longer_than_the_budgets_tiles(in_place):
    need_gpu()
    # their weights take more rounds than a budget of 40 has tiles
    want = check(*scarce(6, [20000, 20000, 15000], 0, page=16, entry=16, layers=1, shared=1250), 40, None, 1, 1, in_place)
    assert want[5] == 2 and want[2].tolist() == [20000, 20000, 40]
