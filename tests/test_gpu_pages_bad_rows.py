"""Rows that are longer than the table is wide, and bad cells, in every row that the page operators read."""
import numpy as np
import pytest

from gpu_util import need_gpu
from test_gpu_pages import check_compact, check_fork, pool

pytestmark = pytest.mark.gpu

LONG = 2 ** 31 - 1


@pytest.mark.parametrize("rows,width,blocks", [(4, 6, 70), (2000, 30, 130001)])
@pytest.mark.parametrize("over", [1, LONG])
def test_compact_flags_rows_longer_than_the_table(rows, width, blocks, over):
    """The status bit; the cells within the table are translated as those of a full row."""
    need_gpu()
    _, cache, table, lens, refs = pool(64, rows=rows, page=2, width=width, blocks=blocks, layers=1)
    r = int(np.argmax(lens))
    n = -(-int(lens[r]) // 2)
    free = np.flatnonzero(refs == 0)[:width - n]
    table[r, n:], refs[free] = free, 1
    lens[r] = 2 * width
    assert check_compact(cache, table, lens, refs)[5] == 0            # exactly full: nothing to flag
    lens[r] = min(LONG, 2 * width + over)
    assert check_compact(cache, table, lens, refs, in_place=True)[5] == 1


def test_compact_flags_rows_of_a_table_without_cells():
    need_gpu()
    _, cache, table, lens, refs = pool(65, rows=3, blocks=40)
    assert check_compact(cache, table[:, :0], np.array([0, -4, 0], np.int32), refs)[5] == 0
    assert check_compact(cache, table[:, :0], np.array([0, 1, 0], np.int32), refs)[5] == 1


@pytest.mark.parametrize("rows,width,blocks", [(4, 6, 70), (2000, 30, 130001)])
@pytest.mark.parametrize("share", [True, False])
def test_fork_flags_rows_that_nobody_descends_from(rows, width, blocks, share):
    """A freed row is read for the references that it gives up: its bad cells and its length are flagged like any row's."""
    need_gpu()
    _, cache, table, lens, refs = pool(66, rows=rows, page=2, width=width, blocks=blocks, layers=1)
    r = int(np.argmax(lens))
    parent = [i for i in range(rows) if i != r]
    assert check_fork(cache, table, lens, refs, parent, share)[4] == 0
    bad = table.copy()
    bad[r, 1] = blocks
    assert check_fork(cache, bad, lens, refs, parent, share)[4] == 1
    bad[r, 1] = -1
    assert check_fork(cache, bad, lens, refs, parent, share, in_place=True)[4] == 1
    n = -(-int(lens[r]) // 2)
    free = np.flatnonzero(refs == 0)[:width - n]
    table[r, n:], refs[free] = free, 1
    lens[r] = 2 * width
    assert check_fork(cache, table, lens, refs, parent, share)[4] == 0
    for over in (2 * width + 1, LONG):
        lens[r] = over
        assert check_fork(cache, table, lens, refs, parent, share)[4] == 1


def test_fork_flags_a_parent_that_finds_no_pages_and_has_a_bad_cell():
    need_gpu()
    _, cache, table, lens, refs = pool(67, rows=3, blocks=60)
    refs[refs == 0] = 1
    table[int(np.argmax(lens)), 0] = 60
    want = check_fork(cache, table, lens, refs, [int(np.argmax(lens))] * 2, False)
    assert want[4] > 0
