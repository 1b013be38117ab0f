"""The oracle of draft verification with negative values, NaN and sums past the range, pinned by hand."""
import numpy as np
import pytest

from oracle import serving


@pytest.mark.parametrize("pd,qd,stands", [(0.0, -0.5, False), (-0.125, -1.0, False), (0.5, np.nan, True), (0.5, -2.0, True),
                                          (np.nan, -1.0, False), (np.nan, 0.5, False), (0.0, np.nan, False), (0.5, 0.5, True)])
def test_negative_values_and_nan_count_as_nothing(pd, qd, stands):
    p, q = np.array([[0.0, pd, 0.5], [0.25, 0.0, 0.0]]), np.array([[0.0, qd, 0.0]])
    out, acc, _, _, bad = serving.verify(p, q, [1], [0, 2], [0.25, 0.5])
    assert acc.tolist() == [int(stands)] and out.tolist() == [[1, 0] if stands else [2, -1]] and bad == 0


def test_sums_past_the_range():
    p = np.array([[2.0 ** 126, 2.0 ** 126], [2.0 ** 126, 2.0 ** 125], [np.inf, 0.0]])
    out, acc, _, _, bad = serving.verify(p, None, [], [0, 1, 2, 3], [0.5, 0.5, 0.5])
    assert out.tolist() == [[-1], [0], [-1]] and acc.tolist() == [0, 0, 0] and bad == 2
