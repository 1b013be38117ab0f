"""Draft verification on the GPU with negative values and NaN among the probabilities, which count as 0 wherever they stand."""
import numpy as np
import pytest

from gpu_util import need_gpu
from test_gpu_verify import check

pytestmark = pytest.mark.gpu


def one(pd, qd, u, bf16=False, V=5):
    """One request with one draft, token 1, whose probabilities are pd and qd -> whether it stands."""
    p, q = np.zeros((2, V), np.float32), np.zeros((1, V), np.float32)
    p[:, 3] = 0.5
    p[0, 1], q[0, 1] = pd, qd
    c = dict(target=p, draft=q, tokens=np.array([1], np.int32), start=np.array([0, 2], np.int32),
             uniform=np.array([u, 0.5], np.float32), greedy=None, seq=np.array([5], np.int32))
    got = check(c, bf16, exact=True)
    return got[0, 1] != -1


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("u", [0.0, 0.25, 0.75])
def test_acceptance(u, bf16):
    need_gpu()
    nan, inf = np.nan, np.inf
    for pd, qd, stands in ((0.0, -0.5, False), (-0.125, -1.0, False), (-0.0, -0.5, False), (0.5, nan, True), (0.5, -2.0, True),
                           (nan, -1.0, False), (nan, nan, False), (-1.0, nan, False), (0.0, nan, False), (0.5, -inf, True),
                           (nan, 0.5, False), (-0.5, 0.5, False), (0.5, 0.5, True), (0.25, 1.0, u < 0.25)):
        assert one(pd, qd, u, bf16) == stands, (pd, qd)


def test_a_draft_without_probabilities():
    need_gpu()
    for pd in (np.nan, -0.5, 0.0, -0.0):
        p = np.array([[0.0, pd, 0.5], [0.5, 0.0, 0.0]], np.float32)
        c = dict(target=p, draft=None, tokens=np.array([1], np.int32), start=np.array([0, 2], np.int32),
                 uniform=np.array([0.0, 0.5], np.float32), greedy=None, seq=np.array([5], np.int32))
        assert check(c, exact=True).tolist() == [[2, -1]]


def test_batches_with_some_of_each():
    need_gpu()
    rng = np.random.default_rng(3)
    V, R, k = 600, 40, 3
    start = (np.arange(R + 1) * (k + 1)).astype(np.int32)
    p = rng.random((R * (k + 1), V)).astype(np.float32)
    q = rng.random((R * k, V)).astype(np.float32)
    for a in (p, q):
        z = rng.random(a.shape)
        a[z < 0.2] *= -1
        a[(z > 0.3) & (z < 0.4)] = np.nan
    c = dict(target=p, draft=q, tokens=rng.integers(0, V, R * k).astype(np.int32), start=start,
             uniform=rng.random(len(p)).astype(np.float32), greedy=None, seq=np.full(R, 9, np.int32))
    check(c)
    check(c, bf16=True)
