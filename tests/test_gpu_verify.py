"""Draft verification on the GPU against the oracle (oracle/serving.py).

Accepted drafts and greedy tokens are equal to the oracle's.  A drawn token is one whose border lies within 2^-44 of the
whole from the wanted sum: sums are held to 2^-46 of themselves.  Where all sums are exact in 64 bits it is the oracle's.
"""
import numpy as np
import pytest
import torch

import sparse_mla_decode_combine_gb300 as pkg
from gpu_util import need_gpu
from oracle import serving

pytestmark = pytest.mark.gpu


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def rows(rng, n, V, sharp=3.0):
    z = rng.standard_normal((n, V)) * sharp
    e = np.exp(z - z.max(1, keepdims=True, initial=0))
    return (e / e.sum(1, keepdims=True)).astype(np.float32)


def batch(seed, ks, V, drafts=True, greedy=0.0, near=0.5):
    rng = np.random.default_rng(seed)
    start = np.concatenate([[0], np.cumsum(np.array(ks) + 1)]).astype(np.int32)
    N, Nd = int(start[-1]), int(sum(ks))
    p = rows(rng, N, V)
    of = np.concatenate([np.arange(start[b], start[b + 1] - 1) for b in range(len(ks))]).astype(int) if Nd else np.zeros(0, int)
    q = p[of] * np.exp(near * rng.standard_normal((Nd, V))).astype(np.float32)
    q = (q / q.sum(1, keepdims=True)).astype(np.float32)
    tok = np.array([rng.choice(V, p=r / r.sum()) for r in q.astype(np.float64)], dtype=np.int32).reshape(Nd)
    g = (rng.random(len(ks)) < greedy).astype(np.uint8)
    for b in np.flatnonzero(g):          # greedy requests' drafts: often the largest value
        d0 = start[b] - b
        for j in range(ks[b]):
            if rng.random() < 0.7:
                tok[d0 + j] = serving.largest(p[start[b] + j])
    return dict(target=p, draft=q if drafts else None, tokens=tok, start=start, uniform=rng.random(N).astype(np.float32),
                greedy=g if greedy else None, seq=rng.integers(20, 90, len(ks)).astype(np.int32))


def to_bf16(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda().bfloat16()


def check(c, bf16=False, gap=0, shift=0, exact=False, status=None, width=None, stream=None):
    """gap: values between rows; shift: values before the first; exact: the oracle's tokens bit for bit."""
    def strided(a):
        if a is None:
            return None
        t = to_bf16(a) if bf16 else dev(a)
        n, V = t.shape
        room = torch.full((shift + n * (V + gap) + 1,), float("nan"), dtype=t.dtype, device="cuda")
        view = room[shift:shift + n * (V + gap)].view(n, V + gap)[:, :V]
        view.copy_(t)
        return view
    p, q = strided(c["target"]), strided(c["draft"])
    R = len(c["start"]) - 1
    W = width or max(int(np.diff(c["start"]).max()), 1)
    full = torch.full((R + 2, W + 1), 77, dtype=torch.int32, device="cuda")
    out, acc, seq = full[1:-1, :W], torch.full((R + 2,), 77, dtype=torch.int32, device="cuda"), dev(c["seq"])
    args = p, q, dev(c["tokens"]), dev(c["start"]), dev(c["uniform"]), out, acc[1:-1], dev(c["greedy"]), seq, seq
    torch.cuda.synchronize()
    pkg.dsv4_get_device_status()
    pkg.check(pkg.dsv4_verify_drafts(*args, stream=stream), "verify")
    torch.cuda.synchronize()
    got_status = pkg.dsv4_get_device_status()
    pn = p.float().cpu().numpy()
    qn = None if q is None else q.float().cpu().numpy()
    want, wacc, wseq, may, bad = serving.verify(pn, qn, c["tokens"], c["start"], c["uniform"], c["greedy"], c["seq"], W)
    got, gacc = out.cpu().numpy(), acc.cpu().numpy()
    assert got_status == (pkg.DSV4_ERR_BAD_INDEX if bad else pkg.DSV4_OK), bad
    assert np.array_equal(gacc[1:-1], wacc) and np.array_equal(seq.cpu().numpy(), wseq)
    for b in range(R):
        a = wacc[b]
        assert np.array_equal(got[b, :a], want[b, :a]) and np.all(got[b, a + 1:] == -1), b
        assert got[b, a] == want[b, a] if exact else got[b, a] in may[b], (b, got[b, a], want[b, a])
    f = full.cpu().numpy()
    assert np.all(f[[0, -1]] == 77) and np.all(f[:, W] == 77) and gacc[0] == gacc[-1] == 77
    return got


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("drafts", [False, True])
@pytest.mark.parametrize("V", [1, 2, 31, 1000, 1024, 1025, 4097, 33001])
def test_batches(V, drafts, bf16):
    need_gpu()
    check(batch(V, [3, 0, 1, 7, 2, 0, 5], V, drafts, greedy=0.3), bf16)


@pytest.mark.parametrize("R,V", [(1, 150001), (1, 8191), (2, 65536), (30, 20000), (80, 9000), (160, 5000), (400, 3000)])
def test_request_counts(R, V):
    need_gpu()
    rng = np.random.default_rng(R)
    check(batch(R, rng.integers(0, 4, R).tolist(), V, greedy=0.2))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("gap,shift", [(1, 0), (3, 1), (8, 4), (0, 7), (5, 2)])
def test_strides_and_alignments(gap, shift, bf16):
    need_gpu()
    check(batch(gap + 10 * shift, [2, 4, 1], 2500, greedy=0.4), bf16, gap, shift)


def test_many_drafts():
    need_gpu()
    check(batch(5, [40, 64, 33, 32, 31], 300, near=0.01), width=70)


def test_draws_on_borders_are_exact():
    need_gpu()
    # equal weights of 2^-13: every sum is exact, and u = i / 8192 lies on the border before token i
    V, R = 8192, 64
    rng = np.random.default_rng(2)
    at = rng.integers(0, V, R)
    c = dict(target=np.full((R, V), 2.0 ** -13, np.float32), draft=None, tokens=np.zeros(0, np.int32),
             start=np.arange(R + 1, dtype=np.int32), uniform=(at / V).astype(np.float32), greedy=None, seq=at.astype(np.int32))
    assert np.array_equal(check(c, exact=True)[:, 0], at)
    # the same with zeros between, in BF16, on a cluster
    c["target"] = np.zeros((1, 2 * 65536), np.float32)
    c["target"][:, 1::2] = 2.0 ** -16
    c.update(start=np.array([0, 1], np.int32), uniform=np.array([12345 / 65536], np.float32), seq=np.array([9], np.int32))
    assert check(c, bf16=True, exact=True)[0, 0] == 2 * 12345 + 1


def test_acceptance_on_borders():
    need_gpu()
    # u q(d) = p(d) is not below it; the next u below is.  Products of 48 bits that fp32 would round together
    q = np.float32(1 + 2.0 ** -23)
    u = np.float32(1 - 2.0 ** -24)
    p = np.float32(float(u) * float(q))      # rounded: 1 + 2^-24 - 2^-47 -> 1
    for pd, stands in ((np.float32(1.0), float(u) * float(q) < 1.0), (np.nextafter(p, np.float32(2), dtype=np.float32), True),
                       (np.nextafter(p, np.float32(0), dtype=np.float32), False), (np.float32(0.5), False)):
        c = dict(target=np.array([[pd, 0.5], [1.0, 0.0]], np.float32), draft=np.array([[q, 0.0]], np.float32),
                 tokens=np.array([0], np.int32), start=np.array([0, 2], np.int32), uniform=np.array([u, 0.5], np.float32),
                 greedy=None, seq=np.array([5], np.int32))
        got = check(c, exact=True)
        assert (got[0, 1] != -1) == stands
    c["uniform"][0], c["draft"][0, 0], c["target"][0, 0] = 0.5, 1.0, 0.5
    assert check(c, exact=True)[0].tolist() == [1, -1]
    c["uniform"][0] = np.nextafter(np.float32(0.5), np.float32(0))
    assert check(c, exact=True)[0].tolist() == [0, 0]


def test_rows_with_nothing_left():
    need_gpu()
    p = np.array([[0.25, 0.0, 0.5], [0, 0, 0], [0.0, 0.75, 0.0], [0, 0, 0], [np.nan, -1.0, 0.0], [np.nan, 0.5, -3.0]], np.float32)
    q = np.array([[0.25, 1.0, 0.5], [1.0, 0.75, 0.0]], np.float32)
    c = dict(target=p, draft=q, tokens=np.array([1, 0], np.int32), start=np.array([0, 2, 4, 5, 6], np.int32),
             uniform=np.full(6, 0.4, np.float32), greedy=None, seq=np.full(4, 8, np.int32))
    assert check(c, exact=True).tolist() == [[2, -1], [1, -1], [-1, -1], [1, -1]]    # p itself where p - q leaves nothing
    c["draft"] = None
    assert check(c, exact=True).tolist() == [[2, -1], [1, -1], [-1, -1], [1, -1]]


def test_greedy_rows_may_be_logits_with_ties_and_infinities():
    need_gpu()
    V = 40000
    rng = np.random.default_rng(4)
    z = rng.integers(-6, 6, (8, V)).astype(np.float32)
    z[1] = -np.inf
    z[2] = np.nan
    z[2, 777] = -np.inf
    z[3, 5] = z[3, 39999] = np.inf
    z[4] = -1.0
    z[4, 100], z[4, 50] = 0.0, -0.0
    z[5] = np.nan
    first = [serving.largest(r) for r in z]
    tok = np.array([first[0], 0, first[2], first[3], 50, 0], np.int32)   # requests of 2, 2 and 2 drafts
    c = dict(target=np.concatenate([z[:3], z[2:5], z[4:5], z[3:5]]), draft=None, tokens=tok, start=np.array([0, 3, 6, 9], np.int32),
             uniform=np.zeros(9, np.float32), greedy=np.ones(3, np.uint8), seq=np.full(3, 60, np.int32))
    assert check(c, exact=True)[1].tolist() == [777, 5, 50]
    c = dict(c, target=z[5:6], tokens=np.zeros(0, np.int32), start=np.array([0, 1], np.int32), uniform=np.zeros(1, np.float32),
             greedy=np.ones(1, np.uint8), seq=np.array([3], np.int32))
    check(c, exact=True)                     # nothing but NaN: -1, and the status bit


def test_bad_requests_and_tokens_are_flagged():
    need_gpu()
    c = batch(6, [2, 1, 3], 500)
    for tok in (-1, 500, 2 ** 31 - 1, -2 ** 31):
        d = dict(c, tokens=c["tokens"].copy())
        d["tokens"][2] = tok
        check(d)
        check(dict(d, draft=None))
    check(dict(c, start=np.array([0, 3, 3, 9], np.int32)), width=6)       # a request without a row
    check(dict(c, start=np.array([0, 3, 5, 10], np.int32)), width=6)      # rows past the last one
    check(dict(c, start=np.array([0, 4, 2, 9], np.int32)), width=6)       # falling
    check(c, width=3)                                                      # more drafts than the output has room for
    check(dict(c, start=c["start"] + 1000))                                # only differences count


def test_a_draft_of_minus_one_never_stands():
    need_gpu()
    z = np.full((3, 5000), np.nan, np.float32)
    z[1:, 7] = 1.0
    for greedy in (None, np.ones(1, np.uint8)):
        got = check(dict(target=z, draft=None, tokens=np.array([-1, 7], np.int32), start=np.array([0, 3], np.int32),
                         uniform=np.zeros(3, np.float32), greedy=greedy, seq=np.array([9], np.int32)), exact=True)
        assert got.tolist() == [[-1, -1, -1]]


def test_bad_tokens_after_the_last_accepted_one_are_flagged():
    need_gpu()
    for greedy in (None, np.ones(2, np.uint8)):
        c = dict(batch(14, [3, 40], 300), greedy=greedy)
        c["uniform"][:] = 0.999999                   # (drafts stand only where the target likes them more)
        c["tokens"][-1] = 300
        check(c)


@pytest.mark.parametrize("u", [1.0, 1.5, -1.0, np.nan, np.inf])
def test_numbers_outside_their_range_draw_some_token(u):
    need_gpu()
    for V, R in ((50, 3), (20000, 1)):
        c = batch(15, [0] * R, V)
        out, acc = torch.empty(R, 1, dtype=torch.int32, device="cuda"), torch.empty(R, dtype=torch.int32, device="cuda")
        uniform = torch.full((R,), u, device="cuda")
        pkg.check(pkg.dsv4_verify_drafts(dev(c["target"]), None, dev(c["tokens"]), dev(c["start"]), uniform, out, acc))
        assert bool(((out >= 0) & (out < V)).all()) and acc.tolist() == [0] * R
        if u >= 1.0:
            assert bool((out == V - 1).all())        # the last one with weight


@pytest.mark.parametrize("R", [1, 500])
def test_the_widest_vocabulary(R):
    need_gpu()
    # one request of 2^22 values; with 500 requests (the others have no rows, and are flagged) one CTA sums them all
    V = 1 << 22
    rng = np.random.default_rng(R)
    p = torch.from_numpy(rng.random((2, V)).astype(np.float32)).cuda()
    q = torch.from_numpy(rng.random((1, V)).astype(np.float32)).cuda()
    start = torch.full((R + 1,), 2, dtype=torch.int32, device="cuda")
    start[0] = 0
    for u in (0.0, 0.37, 0.999):
        p[0, 17], q[0, 17] = 0.0, 0.5                # turned down
        uniform = torch.tensor([0.5, u], device="cuda")
        out, acc = torch.full((R, 2), 9, dtype=torch.int32, device="cuda"), torch.empty(R, dtype=torch.int32, device="cuda")
        tok = torch.tensor([17], dtype=torch.int32, device="cuda")
        pkg.check(pkg.dsv4_verify_drafts(p, q, tok, start, uniform, out, acc))
        pkg.dsv4_get_device_status()
        _, _, _, may, _ = serving.verify(p.cpu().numpy(), q.cpu().numpy(), [17], [0, 2], uniform.cpu().numpy(), width=2)
        assert int(out[0, 0]) in may[0] and int(out[0, 1]) == -1 and bool((out[1:] == -1).all())
        p[0, 17] = 1.0                               # accepted: 0.5 * 0.5 < 1
        pkg.check(pkg.dsv4_verify_drafts(p, q, tok, start, uniform, out, acc))
        pkg.dsv4_get_device_status()
        _, _, _, may, _ = serving.verify(p.cpu().numpy(), q.cpu().numpy(), [17], [0, 2], uniform.cpu().numpy(), width=2)
        assert int(out[0, 0]) == 17 and int(out[0, 1]) in may[0]


def test_rows_past_two_gigabytes():
    need_gpu()
    V, N = 100000, 11000                             # 4.4 GB of float32
    p = torch.zeros(N, V, device="cuda")
    at = torch.randint(0, V, (N,), device="cuda")
    p[torch.arange(N, device="cuda"), at] = 0.25
    start = torch.tensor([0, N - 3, N - 2, N], dtype=torch.int32, device="cuda")
    tok = torch.cat([at[:N - 4], at[N - 2:N - 1]]).int()
    out, acc = torch.empty(3, N, dtype=torch.int32, device="cuda"), torch.empty(3, dtype=torch.int32, device="cuda")
    pkg.check(pkg.dsv4_verify_drafts(p, None, tok, start, torch.full((N,), 0.2, device="cuda"), out, acc))
    assert acc.tolist() == [N - 4, 0, 1]
    want = torch.full((3, N), -1, dtype=torch.int32, device="cuda")
    want[0, :N - 3], want[1, 0], want[2, :2] = at[:N - 3].int(), at[N - 3], at[N - 2:].int()
    assert torch.equal(out, want)
    pkg.check(pkg.dsv4_get_device_status())


def test_empty_calls_and_single_tokens():
    need_gpu()
    e = torch.empty
    i = dict(dtype=torch.int32, device="cuda")
    pkg.check(pkg.dsv4_verify_drafts(e(0, 5, device="cuda"), None, e(0, **i), e(1, **i), e(0, device="cuda"), e(0, 1, **i), e(0, **i)))
    c = batch(8, [0] * 5, 777)
    check(c)
    check(dict(c, draft=None))
    tok, acc = pkg.verify_drafts(dev(c["target"]), None, dev(c["tokens"]), dev(c["start"]), dev(c["uniform"]), 0)
    assert tok.shape == (5, 1) and acc.tolist() == [0] * 5


def test_refusals():
    need_gpu()
    c = batch(9, [1, 2], 64)
    p, q, t, s, u = (dev(c[k]) for k in ("target", "draft", "tokens", "start", "uniform"))
    out, acc = torch.empty(2, 3, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        pkg.dsv4_verify_drafts(p.half(), None, t, s, u, out, acc)
    with pytest.raises(TypeError):
        pkg.dsv4_verify_drafts(p, q.bfloat16(), t, s, u, out, acc)
    with pytest.raises(TypeError):
        pkg.dsv4_verify_drafts(p, q, t.long(), s, u, out, acc)
    with pytest.raises(ValueError):
        pkg.dsv4_verify_drafts(p, q[:2], t, s, u, out, acc)
    with pytest.raises(ValueError):
        pkg.dsv4_verify_drafts(p, q, t, s[:2], u, out, acc)
    with pytest.raises(ValueError):
        pkg.dsv4_verify_drafts(p.cpu(), q, t, s, u, out, acc)
    with pytest.raises(ValueError):
        pkg.dsv4_verify_drafts(p.t().contiguous().t(), q, t, s, u, out, acc)
    assert pkg.dsv4_verify_drafts(p, q, t, s, u, out, acc, None, acc) == pkg.DSV4_ERR_INVALID_ARG


def test_streams_and_graphs():
    need_gpu()
    c = batch(11, [3, 1, 0, 2], 30000, greedy=0.25)
    side = torch.cuda.Stream()
    check(c, stream=side)
    p, q, t, s, u, g = (dev(c[k]) for k in ("target", "draft", "tokens", "start", "uniform", "greedy"))
    out, acc = torch.empty(4, 4, dtype=torch.int32, device="cuda"), torch.empty(4, dtype=torch.int32, device="cuda")
    pkg.check(pkg.dsv4_verify_drafts(p, q, t, s, u, out, acc, g))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkg.check(pkg.dsv4_verify_drafts(p, q, t, s, u, out, acc, g))
        pkg.check(pkg.dsv4_verify_drafts(p, q, t, s, u, out, acc, g))
    for seed in (1, 2):
        new = np.random.default_rng(seed).random(len(c["uniform"])).astype(np.float32)
        u.copy_(dev(new))
        out.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        _, wacc, _, may, _ = serving.verify(c["target"], c["draft"], c["tokens"], c["start"], new, c["greedy"])
        assert acc.tolist() == wacc.tolist() and all(int(out[b, wacc[b]]) in may[b] for b in range(4))
