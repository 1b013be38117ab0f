"""The page operators on a table that has rows but no cells (max_blocks 0): every row is empty."""
import numpy as np
import pytest

from gpu_util import need_gpu
from test_gpu_pages import check_compact, check_fork, pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1, 3])
def test_tables_without_cells(rows):
    need_gpu()
    _, cache, table, _, _ = pool(65, rows=rows, blocks=40)
    lens, refs = np.zeros(rows, np.int32), np.zeros(40, np.int32)
    refs[[3, 20]] = 1, 2                                              # pages of another holder
    check_fork(cache, table[:, :0], lens, refs, [0, -1, rows - 1, 0], True)
    check_fork(cache, table[:, :0], lens, refs, [0] * rows, False, in_place=True)
    want = check_compact(cache, table[:, :0], lens, refs)
    assert want[4] == 2 and want[5] == 0
