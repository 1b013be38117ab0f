"""Rows that are longer than the table is wide, and bad cells, in every row that the page operators read."""
import numpy as np
import pytest

from gpu_util import need_gpu
from test_gpu_pages import check_compact, pool

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
