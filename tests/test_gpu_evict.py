"""Eviction on the GPU against the oracle (oracle/serving.py): every byte, table cell, length, count and weight."""
import numpy as np
import pytest
import torch

import sparse_mla_decode_combine_gb300 as pkg
from gpu_util import need_gpu
from oracle import serving

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def pool(seed, lens, page=4, width=None, spare=4, layers=2, entry=16, shared=0, ties=False):
    """Rows of the given lengths in scattered pages; rows 2i and 2i + 1 share their first `shared` pages."""
    rng = np.random.default_rng(seed)
    lens = np.array(lens, np.int32)
    n = -(-lens // page)
    width = int(max(1, n.max(initial=1))) if width is None else width
    blocks = int(n.sum()) + spare
    table, perm, at = np.full((len(lens), width), -1, np.int32), rng.permutation(blocks), 0
    for r in range(len(lens)):
        s = min(shared, n[r], n[r - 1]) if r % 2 else 0
        table[r, :s] = table[r - 1, :s]
        table[r, s:n[r]] = perm[at:at + n[r] - s]
        at += n[r] - s
    refs = np.bincount(table[table >= 0], minlength=blocks).astype(np.int32)
    cache = rng.integers(0, 256, (layers, blocks, page, entry)).astype(np.uint8)
    w = np.exp(2 * rng.standard_normal((len(lens), width * page))).astype(np.float32)
    if ties:
        w = np.floor(w * 2) / 2
    w[np.arange(width * page) >= lens[:, None]] = 0
    return cache, table, lens, refs, w.astype(np.float32)


def check(cache, table, lens, refs, w, budget, limit=None, first=0, recent=0, in_place=False, status=None, stream=None, gap=3,
          wide=5):
    limit = budget if limit is None else limit
    want = serving.evict(cache, table, lens, refs, w, budget, limit, first, recent)
    (R, M), (L, B, page, entry) = table.shape, cache.shape
    c, r = dev(cache), dev(refs)
    t_in = torch.full((R, M + 2), 2 ** 30, dtype=torch.int32, device="cuda")
    t_in[:, :M] = dev(table)
    t_out = torch.full((R + 2, M + 1), 77, dtype=torch.int32, device="cuda")
    l_out = torch.full((R + 2,), 77, dtype=torch.int32, device="cuda")
    w_in = torch.full((R, M * page + wide + gap), 7.0, device="cuda")
    w_in[:, :M * page], w_in[:, M * page:M * page + wide] = dev(w), 0
    w_out = w_in if in_place else torch.full((R + 2, M * page + wide + gap), 7.0, device="cuda")
    r_out = r if in_place else torch.full_like(r, 77)
    ws = pkg.workspace_for_cache_evict(R, M, B, L, page, entry, budget)
    ws.fill_(0xA5)
    wv = (w_in if in_place else w_out[1:-1])[:, :M * page + wide]
    torch.cuda.synchronize()
    pkg.dsv4_get_device_status()
    pkg.check(pkg.dsv4_cache_evict(c, t_in[:, :M], dev(lens), r, w_in[:, :M * page + wide], budget, limit, first, recent,
                                   t_out[1:-1, :M], l_out[1:-1], r_out, wv, ws, stream), "evict")
    torch.cuda.synchronize()
    st = pkg.dsv4_get_device_status()
    assert st == (pkg.DSV4_ERR_BAD_INDEX if want[5] else pkg.DSV4_OK), want[5]
    assert np.array_equal(l_out.cpu().numpy()[1:-1], want[2])
    assert np.array_equal(t_out.cpu().numpy()[1:-1, :M], want[1])
    assert np.array_equal(r_out.cpu().numpy(), want[3])
    got_w = wv.cpu().numpy()
    assert np.array_equal(got_w[:, :M * page].view(np.uint32), want[4].view(np.uint32)) and not got_w[:, M * page:].any()
    assert np.array_equal(c.cpu().numpy(), want[0])
    f = t_out.cpu().numpy()
    assert np.all(f[[0, -1]] == 77) and np.all(f[:, M] == 77) and l_out[0] == 77 and l_out[-1] == 77
    assert bool((w_in[:, M * page + wide:] == 7).all()) and bool((w_out[:, M * page + wide:] == 7).all())
    return want


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("budget,limit,first,recent", [(10, 10, 0, 0), (10, 14, 3, 2), (10, 10, 10, 0), (10, 10, 0, 10), (1, 1, 0, 0),
                                                       (1, 1, 1, 0), (12, 12, 4, 4), (16, 20, 5, 11), (29, 29, 1, 1)])
def test_small_rows(budget, limit, first, recent, in_place):
    need_gpu()
    lens = [0, 1, 9, 10, 11, 13, 14, 15, 30, 29, 28, 31]
    check(*pool(budget, lens), budget, limit, first, recent, in_place)
    check(*pool(budget, lens, ties=True), budget, limit, first, recent, in_place)


@pytest.mark.parametrize("shared", [1, 3, 100])
@pytest.mark.parametrize("budget,first,recent", [(12, 4, 2), (13, 8, 0), (16, 16, 0), (7, 0, 7), (20, 0, 0)])
def test_shared_pages(budget, first, recent, shared):
    need_gpu()
    lens = [30, 30, 25, 31, 40, 8, 3, 40, 40, 40]
    check(*pool(shared, lens, shared=shared, spare=30), budget, None, first, recent)
    check(*pool(shared, lens, shared=shared, spare=30), budget, budget + 12, first, recent, in_place=True)


@pytest.mark.parametrize("spare", [0, 1, 2, 3, 5, 8])
def test_too_few_free_pages(spare):
    need_gpu()
    lens = [30, 30, 25, 31, 24, 24, 40, 9, 40, 40]
    want = check(*pool(2, lens, shared=6, spare=spare), 9, None, 1, 1)
    assert want[5] == (0 if spare >= 27 else want[5])


@pytest.mark.parametrize("page,entry,layers", [(1, 16, 1), (3, 48, 2), (16, 400, 3), (32, 656, 2), (64, 400, 1), (7, 4112, 2),
                                               (2, 32768, 1), (2, 32784, 2), (1, 70000, 1)])
def test_pages_and_entries(page, entry, layers):
    need_gpu()
    n = 40 * page if entry < 4000 else 12 * page
    lens = [n, n - 1, n // 2 + 1, 3, n // 3]
    check(*pool(page, lens, page=page, entry=entry, layers=layers, shared=2, spare=60), max(3, n // 3), None, min(2, n // 4), min(3, n // 5))


@pytest.mark.parametrize("n,budget,first,recent", [(9000, 8999, 4, 100), (9000, 8000, 0, 0), (9000, 3001, 64, 1000),
                                                   (9000, 17, 1, 1), (20011, 12345, 5, 7), (9000, 4096, 4096, 0), (9000, 4096, 0, 4096)])
def test_long_rows_in_place(n, budget, first, recent):
    need_gpu()
    # tiles that wait for one another, through every distance that entries move
    for seed in range(3):
        check(*pool(seed, [n, n - 777, budget + 1], page=16, entry=400, layers=2), budget, None, first, recent, in_place=seed == 1)


@pytest.mark.parametrize("n,budget,first,recent", [(70001, 30000, 3, 500), (131072 + 40, 131000, 17, 23), (131072 + 64, 20000, 0, 1),
                                                   (150001, 60000, 5, 999)])
@pytest.mark.parametrize("ties", [False, True])
def test_rows_of_many_entries(n, budget, first, recent, ties):
    need_gpu()
    cache, table, lens, refs, w = pool(budget, [n, 100, n - 5000], page=64, entry=16, layers=1, ties=ties)
    if ties:
        w[:, ::3] = 0
    check(cache, table, lens, refs, w, budget, None, first, recent, in_place=ties)


def test_thresholds_of_every_kind():
    need_gpu()
    cache, table, lens, refs, w = pool(12, [2000] * 6, page=16, entry=16, layers=1)
    i = np.arange(w.shape[1])
    w[0] = np.where(i % 2, 1.0, np.nextafter(np.float32(1), np.float32(2)))       # keys that differ in their last bit
    w[1] = -1.0 - i                                                               # below 0
    w[2] = np.where(i < 1500, 0.0, 5.0)                                           # 0 is the threshold
    w[3] = np.where(i < 300, np.inf, np.where(i < 500, -np.inf, np.nan))          # NaN is the threshold
    w[4] = np.float32(1e-45) * (i % 7)                                            # subnormal ones
    w[5] = np.finfo(np.float32).max
    w = w.astype(np.float32)
    for budget in (1000, 777, 1999):
        check(cache, table, lens, refs, w.copy(), budget, None, 2, 5)


def test_one_entry_leaves_a_long_row():
    need_gpu()
    cache, table, lens, refs, w = pool(3, [6000, 6000, 6000], page=64, entry=64, layers=3)
    for at in (0, 3000, 5999):
        w[:] = 1 + np.arange(w.shape[1])[::-1] % 7
        w[:, at] = 0
        check(cache, table, lens, refs, w, 5999)


def test_weights_with_ties_infinities_and_nan():
    need_gpu()
    rng = np.random.default_rng(4)
    cache, table, lens, refs, w = pool(4, [3000, 2500, 2000, 700], page=16, entry=16)
    w = rng.choice(np.array([0.0, -0.0, 1.0, 2.0, np.inf, -np.inf, np.nan, -1.0], np.float32), w.shape)
    w[0] = 0.0
    w[3, :600] = np.nan
    for budget, first, recent in ((1000, 4, 64), (650, 0, 0), (1999, 1, 0)):
        check(cache, table, lens, refs, w.copy(), budget, None, first, recent)


def test_many_rows():
    need_gpu()
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 60, 3000)
    check(*pool(5, lens, page=4, layers=1, shared=2, spare=9000), 20, 25, 2, 5)


def test_bad_pages_and_lengths():
    need_gpu()
    cache, table, lens, refs, w = pool(6, [30, 30, 30, 30, 30, 12], spare=8)
    t = table.copy()
    t[0, 0], t[1, 3], t[2, 7], t[5, 1] = -1, len(refs), 2 ** 31 - 1, -5
    check(cache, t, lens, refs, w, 11, None, 2, 3)
    s = lens.copy()
    s[0], s[1], s[3] = 2 ** 31 - 1, -2 ** 31, 40
    check(cache, table, np.minimum(s, 2 ** 31 - 1), refs, np.where(w == 0, 0.5, w).astype(np.float32), 11, None, 2, 3)


def test_rows_and_pools_that_are_empty():
    need_gpu()
    check(*pool(7, [0, 0, 0]), 5)
    check(*pool(7, [3, 2, 5]), 5)
    cache, table, lens, refs, w = pool(7, [9, 9])
    check(cache, table[:0], lens[:0], refs, w[:0], 5)
    check(cache, table[:, :0], np.zeros(2, np.int32), refs, w[:, :0], 5)
    check(cache[:, :0], np.full((2, 3), -1, np.int32), np.zeros(2, np.int32), refs[:0], np.zeros((2, 12), np.float32), 5)


def test_layers_apart():
    need_gpu()
    cache, table, lens, refs, w = pool(8, [300, 200, 40], page=16, entry=48, layers=3)
    L, B, page, entry = cache.shape
    room = torch.zeros(L, B + 3, page, entry, dtype=torch.uint8, device="cuda")
    room[:, :B] = dev(cache)
    room[:, B:] = 9
    t, n, r, wt = pkg.cache_evict(room[:, :B], dev(table), dev(lens), dev(refs), dev(w), 100, None, 4, 20, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    want = serving.evict(cache, table, lens, refs, w, 100, 100, 4, 20)
    assert np.array_equal(room[:, :B].cpu().numpy(), want[0]) and bool((room[:, B:] == 9).all())
    for got, ref in zip((t, n, r, wt), want[1:]):
        assert np.array_equal(got.cpu().numpy(), ref)


def test_offsets_past_two_gigabytes():
    need_gpu()
    # one row over pages at both ends of a pool of 2.6 GB a layer
    B, page, entry = 100_000, 64, 400
    rng = np.random.default_rng(9)
    c = torch.randint(0, 256, (1, B, page, entry), dtype=torch.uint8, device="cuda")
    cells = np.concatenate([rng.permutation(50), B - 1 - rng.permutation(50)]).astype(np.int32)[rng.permutation(100)]
    table, lens = cells[None], np.array([6390], np.int32)
    refs = np.zeros(B, np.int32)
    refs[cells] = 1
    w = np.exp(rng.standard_normal((1, 6400))).astype(np.float32)
    small = c[:, torch.from_numpy(cells.astype(np.int64)).cuda()].cpu().numpy()
    want = serving.evict(small, np.arange(100, dtype=np.int32)[None], lens, np.ones(100, np.int32), w, 3000, 3000, 4, 100)
    t, n, r, wt = pkg.cache_evict(c, dev(table), dev(lens), dev(refs), dev(w), 3000, None, 4, 100)
    torch.cuda.synchronize()
    assert np.array_equal(c[:, torch.from_numpy(cells.astype(np.int64)).cuda()].cpu().numpy(), want[0])
    assert np.array_equal(t.cpu().numpy()[0, :47], cells[:47]) and int(r.sum()) == 47 and np.array_equal(wt.cpu().numpy(), want[4])


def test_graph_replays_evict_again():
    need_gpu()
    cache, table, lens, refs, w = pool(10, [900, 700, 650], page=16, entry=400, shared=3, spare=40)
    args = dev(table), dev(lens), dev(refs), dev(w)
    c = dev(cache)
    outs = [torch.empty_like(a) for a in args]
    ws = pkg.workspace_for_cache_evict(*table.shape, len(refs), 2, 16, 400, 300)
    call = lambda: pkg.check(pkg.dsv4_cache_evict(c, *args, 300, 300, 4, 64, outs[0], outs[1], outs[2], outs[3], ws))  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in (1, 2):
        new = np.exp(np.random.default_rng(seed).standard_normal(w.shape)).astype(np.float32)
        args[3].copy_(dev(new))
        c.copy_(dev(cache))
        graph.replay()
        torch.cuda.synchronize()
        want = serving.evict(cache, table, lens, refs, new, 300, 300, 4, 64)
        assert np.array_equal(c.cpu().numpy(), want[0])
        for got, ref in zip(outs, want[1:]):
            assert np.array_equal(got.cpu().numpy(), ref)
    pkg.check(pkg.dsv4_get_device_status())


def test_two_streams_and_other_work_at_once():
    need_gpu()
    # tiles wait for one another while other kernels take multiprocessors
    pools = [pool(20 + i, [20000, 9000, 5000], page=64, entry=400, layers=2) for i in range(2)]
    want = [serving.evict(*c, 3000, 3000, 4, 100) for c in pools]
    state = [[dev(a) for a in c] for c in pools]
    streams = [torch.cuda.Stream() for _ in range(3)]
    a = torch.randn(2048, 2048, device="cuda").bfloat16()
    torch.cuda.synchronize()
    for turn in range(5):
        got = []
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                c = state[i][0].clone()
                got.append((c, pkg.cache_evict(c, *state[i][1:], 3000, None, 4, 100)))
        with torch.cuda.stream(streams[2]):
            for _ in range(20):
                a @ a
        torch.cuda.synchronize()
        for (c, rest), ref in zip(got, want):
            assert np.array_equal(c.cpu().numpy(), ref[0])
            assert all(np.array_equal(x.cpu().numpy(), y) for x, y in zip(rest, ref[1:]))
    pkg.check(pkg.dsv4_get_device_status())


def test_rows_and_pages_given_back_are_taken_by_a_later_call():
    need_gpu()
    cache, table, lens, refs, w = pool(13, [40, 40, 36, 40], shared=5, spare=14)
    args = [cache, table, lens, refs, w]
    d = [dev(a) for a in args]
    for budget in (23, 17, 9, 3):
        want = serving.evict(*args, budget, budget, 1, 2)
        assert want[5] == 0
        d[1:] = list(pkg.cache_evict(*d, budget, None, 1, 2))
        torch.cuda.synchronize()
        assert all(np.array_equal(x.cpu().numpy(), y) for x, y in zip(d, want))
        args = list(want[:5])
        live = args[1][args[1] >= 0]
        assert np.array_equal(np.bincount(live, minlength=len(refs)), args[3])
    pkg.check(pkg.dsv4_get_device_status())


def test_refusals():
    need_gpu()
    cache, table, lens, refs, w = (dev(a) for a in pool(11, [30, 20]))
    outs = [torch.empty_like(a) for a in (table, lens, refs, w)]
    ws = pkg.workspace_for_cache_evict(*table.shape, len(refs), 2, 4, 16, 9)
    f = lambda **kw: pkg.dsv4_cache_evict(**{**dict(  # noqa: E731
        cache=cache, block_table=table, seq_lens=lens, ref_counts=refs, weights=w, budget=9, limit=9, first=1, recent=1,
        block_table_out=outs[0], seq_lens_out=outs[1], ref_counts_out=outs[2], weights_out=outs[3], workspace=ws), **kw})
    for bad in (dict(budget=0), dict(limit=8), dict(first=-1), dict(recent=-1), dict(first=9), dict(recent=9),
                dict(block_table_out=table), dict(seq_lens_out=lens), dict(workspace=ws[:-256])):
        assert f(**bad) == pkg.DSV4_ERR_INVALID_ARG, bad
    with pytest.raises(ValueError):
        f(weights=w[:1])
    with pytest.raises(ValueError):
        f(block_table_out=outs[0][:, :2])
    with pytest.raises(ValueError):
        f(cache=cache[:, ::2])
    with pytest.raises(TypeError):
        f(weights=w.double(), weights_out=outs[3].double())
    with pytest.raises(ValueError):
        f(seq_lens=lens.cpu())
