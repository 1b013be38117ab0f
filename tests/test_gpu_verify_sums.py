"""The accuracy of draft verification's sums on the GPU, where it is hardest: rows of a likely token and a flat tail.

Every value is a multiple of 2^-49 and the whole is below 1, so that sums are exact in 64 bits and the
wanted sum u T in 73: a row is set up to have a border 2^-39 (2^-40 in the smaller vocabularies) of the whole above or below its
wanted sum.  The kernel's sums are within 2^-40 of themselves: with v = 2^-24, half a step of fp32, and an addition of two pairs
good to 3 v^2 of their sum,
  26 v^2       a group of 16 values (8 with a draft): the roundings of the additions' residuals;
  3 v^2        a group joining a lane's sum: up to 16 (32) in the widest vocabularies, 4 (8) up to 2048 values a tile;
  15 v^2       the lanes of a tile;
  48 v^2       the tiles of a lane's run, 16 of them in the widest vocabularies (9 v^2 for the three tiles of 151937 values);
  15 v^2, 9 v^2  the runs, and the CTAs;
  42 v^2       the values before one in its tile, on top of what lies before the tile;
in all 203 v^2 (251 v^2 with a draft) in the widest vocabularies and 128 v^2 (140 v^2) in the smaller, and 3 v^2 of the product u T,
whose sum does without the 42.  Border and wanted sum come near to within both of it: at most 463 v^2 of the whole, below 2^-39, and 241 v^2,
below 2^-40.
"""
import numpy as np
import pytest
import torch

import sparse_mla_decode_combine_gb300 as pkg
from gpu_util import need_gpu
from test_gpu_verify import dev

pytestmark = pytest.mark.gpu


def peaked(V, log_distance, side, at, draft):
    """-> (w, m, token): weights (in units of 2^-49) with a peak of 0.5 at index 0, another at the end, and a flat tail, whose border
    near `at` lies 2^log_distance of the whole above (side 1) or below (side -1) the wanted sum m 2^-24 T, so that `token` is drawn."""
    low = 41 if V > 2 ** 20 else 43          # the tail's values lose as much as they can below 2^-low
    x = (int(2.0 ** -25.5 * 2 ** low) + 0.4375) * 2 ** (49 - low)
    assert x == int(x) and x % 2 == 0
    w = np.full(V, int(x), np.int64)
    w[0], w[-1] = 2 ** 48 + 2 ** 39, 0
    if draft:
        w[7] = 0                             # the drafted token: what it had is taken off
    w[-1] = (2 ** 49 - int(w.sum()) - 2 ** 43) // 2 ** 26 * 2 ** 26
    before, T = int(w[:at].sum()), int(w.sum())
    m = round(before * 2 ** 24 / T)
    # n more among the first values move the border by n (1 - u)
    n = round((side * 2.0 ** log_distance * T - (before - m * T / 2 ** 24)) / (1 - m / 2 ** 24)) // 2 * 2
    each = n // 64 // 2 * 2
    w[8:72] += each
    w[8] += n - 64 * each
    before, T = int(w[:at].sum()), int(w.sum())
    off = (before * 2 ** 24 - m * T) / (T * 2 ** 24)                          # (the difference is exact)
    assert T < 2 ** 49 and 0.98 < side * off * 2.0 ** -log_distance < 1.02 and w[8:72].max() < 2 ** 24
    return w, m, at if side < 0 else at - 1


def draw(p, q, tokens, m, R):
    """What the only request with rows (the first of R) draws with the number m 2^-24."""
    out, acc = torch.full((R, 2), 9, dtype=torch.int32, device="cuda"), torch.empty(R, dtype=torch.int32, device="cuda")
    start = torch.full((R + 1,), len(p), dtype=torch.int32, device="cuda")
    start[0] = 0
    uniform = torch.full((len(p),), 0.75, device="cuda")
    uniform[-1] = m / 2 ** 24
    pkg.check(pkg.dsv4_verify_drafts(dev(p), q if q is None else dev(q), dev(np.array(tokens, np.int32)), start, uniform, out, acc))
    pkg.dsv4_get_device_status()             # (the requests without rows are flagged)
    assert int(acc[0]) == 0 and int(out[0, 1]) == -1
    return int(out[0, 0])


SIZES = [(1 << 22, -39), (151937, -40), (30011, -40)]


@pytest.mark.parametrize("R", [1, 500])      # (with 500 one CTA sums a row, in tiles of up to 8192 values)
@pytest.mark.parametrize("V,log_distance", SIZES)
def test_peaked_rows(V, log_distance, R):
    need_gpu()
    for at in (V // 5, V // 2 + 3, V - V // 7):
        for side in (-1, 1):
            w, m, token = peaked(V, log_distance, side, at, False)
            p = (w * 2.0 ** -49).astype(np.float32)
            assert np.array_equal(p.astype(np.float64) * 2 ** 49, w)
            assert draw(p[None], None, [], m, R) == token, (at, side)


@pytest.mark.parametrize("R", [1, 500])
@pytest.mark.parametrize("V,log_distance", SIZES)
def test_peaked_differences(V, log_distance, R):
    need_gpu()
    for at in (V // 5, V // 2 + 3, V - V // 7):
        for side in (-1, 1):
            w, m, token = peaked(V, log_distance, side, at, True)
            p, q = np.zeros((2, V), np.float32), np.zeros((1, V), np.float32)
            q[0] = np.where(w < 2 ** 26, 2.0 ** -26, 0.0)
            p[0] = w * 2.0 ** -49 + q[0]
            q[0, 7] = 0.5                    # turned down: 0.75 0.5 is not below p(7)
            assert np.array_equal(np.maximum(p[0].astype(np.float64) - q[0], 0) * 2 ** 49, w)
            assert draw(p, q, [7], m, R) == token, (at, side)
