"""The page operators at the sizes where the plan by one CTA gives way to the plan by a cluster: the same state either way."""
import numpy as np
import pytest

from gpu_util import need_gpu
from test_gpu_pages import check_compact, check_copy, check_fork, pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,rows_out,width,blocks", [
    (128, 128, 9, 3000), (128, 129, 9, 3000), (129, 128, 9, 3000), (129, 131, 9, 3000), (64, 64, 256, 9000), (64, 64, 257, 9000),
    (5, 1024, 4, 2000), (1024, 7, 4, 6000), (6, 40, 8, 16384), (6, 40, 8, 16385)])
@pytest.mark.parametrize("share", [True, False])
def test_fork(rows, rows_out, width, blocks, share):
    need_gpu()
    rng, *state = pool(110 + rows, rows=rows, page=2, width=width, blocks=blocks, layers=1, fill=0.5)
    check_fork(*state, rng.integers(-1, rows, rows_out), share, in_place=rows % 2 == 0)


@pytest.mark.parametrize("blocks", [1, 1023, 1024, 1025, 16383, 16384, 16385, 16391])
def test_compact(blocks):
    need_gpu()
    rng, cache, table, lens, refs = pool(111, rows=min(5, blocks // 8), page=2, width=4, blocks=blocks, layers=1)
    spare = np.flatnonzero(refs == 0)
    refs[spare[rng.random(len(spare)) < 0.4]] = 3
    check_compact(cache, table, lens, refs, in_place=blocks % 2 == 0)


@pytest.mark.parametrize("layers,n", [(8, 256), (9, 227), (9, 228), (8, 257), (2049, 1), (1, 256)])
@pytest.mark.parametrize("page", [1, 1025])
@pytest.mark.parametrize("one_pool", [True, False])
def test_copies(layers, n, page, one_pool):
    """Short lists with and without a plan; targets that are named twice, sources that are targets, pages out of range."""
    need_gpu()
    rng = np.random.default_rng(layers + n)
    blocks = 300 if page == 1 else 30
    dst = rng.integers(0, 256, (min(layers, 100) if page > 1 else layers, blocks, page, 16)).astype(np.uint8)
    src = dst if one_pool else rng.integers(0, 256, dst.shape).astype(np.uint8)
    s, d = rng.integers(-1, blocks + 1, n), rng.integers(0, blocks + 1, n)
    check_copy(dst, src, s, d, one_pool)
