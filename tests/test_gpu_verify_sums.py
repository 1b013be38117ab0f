"""The accuracy of draft verification's sums on the GPU, where it is hardest: rows of a likely token and a flat tail, sums of subnormal
values, and sums past the range.

In the peaked rows every value is a multiple of 2^-49 and the whole is below 1, so that sums are exact in 64 bits and the
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
from test_gpu_verify import check, dev

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


def rows(p, u, **over):
    R = len(p)
    return dict(target=p.astype(np.float32), draft=None, tokens=np.zeros(0, np.int32), start=np.arange(R + 1, dtype=np.int32),
                uniform=np.asarray(u, np.float32), greedy=None, seq=np.arange(R, dtype=np.int32) + 5, **over)


@pytest.mark.parametrize("V", [3, 700, 40000])
@pytest.mark.parametrize("log", [-149, -130, -105, -70, -63])
def test_small_sums(V, log):
    need_gpu()
    # whole numbers times a power of 2: sums are exact, and the product with u in 64 bits of fraction
    R = 12
    rng = np.random.default_rng(V - log)
    p = np.ldexp(rng.integers(0, 4, (R, V)).astype(np.float64), log)
    p[:, 0] = np.ldexp(1.0, log)
    u = rng.random(R).astype(np.float32)
    total = np.ldexp(p, -log).sum(1)
    for r in range(R // 2):                  # on a border, or next to one
        u[r] = np.float32(np.float32(rng.integers(0, total[r])) / np.float32(total[r]))
    u[R - 1] = 0.0
    check(rows(p, u), exact=True)


def test_small_differences():
    need_gpu()
    V = 5000
    rng = np.random.default_rng(5)
    q = np.ldexp(rng.integers(0, 9, (1, V)).astype(np.float64), -149).astype(np.float32)
    p = np.concatenate([q + np.ldexp(rng.integers(0, 3, (1, V)).astype(np.float64), -149), q]).astype(np.float32)
    p[0, 9], q[0, 9] = 0.0, 1.0              # turned down
    for u in (0.0, 0.25, 0.5, 0.75, 0.9999):
        check(dict(target=p, draft=q, tokens=np.array([9], np.int32), start=np.array([0, 2], np.int32),
                   uniform=np.array([0.5, u], np.float32), greedy=None, seq=np.array([7], np.int32)), exact=True)


@pytest.mark.parametrize("V", [2, 3000, 50000])
def test_sums_past_the_range_are_flagged(V):
    need_gpu()
    p = np.zeros((6, V), np.float32)
    p[0, :2] = 3e38                          # past fp32's range
    p[1, :2] = 2.0 ** 126                    # 2^127
    p[2, 0], p[2, 1] = 2.0 ** 126, 2.0 ** 125
    p[3, 1] = np.inf
    p[4, 0], p[4, 1] = -3e38, 1e38
    p[5] = 2e38
    got = check(rows(p, [0.75, 0.5, 0.7, 0.5, 0.5, 0.1]), exact=True)
    assert got[:5, 0].tolist() == [-1, -1, 1, -1, 1] and got[5, 0] == -1
    q = np.zeros((1, V), np.float32)
    q[0, 0] = 1e38
    c = dict(target=np.stack([p[0], p[2]]), draft=q, tokens=np.array([0], np.int32), start=np.array([0, 2], np.int32),
             uniform=np.array([np.nan, 0.5], np.float32), greedy=None, seq=np.array([7], np.int32))
    assert check(c, exact=True)[0].tolist() == [-1, -1]
    c["uniform"][0] = 0.5                    # accepted
    assert check(c, exact=True)[0].tolist() == [0, 0]
