"""The oracle of eviction where there are too few free pages, pinned by a case worked out by hand."""
import numpy as np

from oracle import serving


def test_rows_that_find_no_page_stay():
    # pages of 2; rows 0 and 1 share pages 0 and 1, row 2 is alone.  A budget of 3 keeps entries (0, 2, 4), (0, 1, 4), (1, 2, 3): pages 0 and
    # 1 of row 0 are written, so it takes two; page 0 of row 1 stays as it is and page 1 is written, so it takes one
    table, lens = np.array([[0, 1, 2], [0, 1, 3], [4, 5, -1]], np.int32), np.array([5, 5, 4], np.int32)
    cache = np.arange(8, dtype=np.uint8)[None, :, None, None] * 2 + np.arange(2, dtype=np.uint8)[None, None, :, None]
    weights = np.array([[5, 0, 4, 1, 9, 0], [5, 4, 0, 1, 9, 0], [0, 1, 2, 3, 0, 0]], np.float32)
    for free, lengths, bad in (([6, 7], [3, 5, 3], 1), ([7], [5, 5, 3], 2), ([], [5, 5, 3], 2)):
        refs = np.array([2, 2, 1, 1, 1, 1, 1, 1], np.int32)
        refs[free] = 0
        c, t, n, r, w, b = serving.evict(cache, table, lens, refs, weights, 3, 3, 0, 1)
        assert n.tolist() == lengths and b == bad
        for i in (0, 1):
            if lengths[i] == 5:
                assert t[i].tolist() == table[i].tolist() and w[i].tolist() == weights[i].tolist()
        # (row 1 asks for the page after those that row 0 asked for, whether it got them or not)
        assert t[2].tolist() == [4, 5, -1] and w[2].tolist() == [1, 2, 3, 0, 0, 0] and c[0, 4:6, :, 0].tolist() == [[9, 10], [11, 11]]
        if not free[1:]:
            assert r.tolist() == refs.tolist() and np.array_equal(c[0, :4], cache[0, :4])
        else:
            assert t[0].tolist() == [6, 7, -1] and r.tolist() == [1, 1, 0, 1, 1, 1, 1, 1]
            assert c[0, 6:8, 0, 0].tolist() == [0, 4] and c[0, 6, 1, 0] == 2 and w[0].tolist() == [5, 4, 9, 0, 0, 0]
