"""The page operators on the GPU against the oracle (oracle/fp4.py): every byte, table cell, length and count."""
import numpy as np
import pytest
import torch

import sparse_mla_decode_combine_gb300 as pkg
import synth
from gpu_util import need_gpu
from oracle import fp4

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def pool(seed, rows, page=4, width=6, blocks=64, layers=2, entry=16, fill=1.0):
    """Rows of random lengths; row 2i + 1 shares the full pages that it has in common with row 2i."""
    rng = np.random.default_rng(seed)
    lens = (rng.integers(0, width * page + 1, rows) * fill).astype(np.int32)
    table, perm, at = np.full((rows, width), -1, np.int32), rng.permutation(blocks), 0
    for r in range(rows):
        n = -(-int(lens[r]) // page)
        s = min(int(lens[r]), int(lens[r - 1])) // page if r % 2 else 0
        table[r, :s] = table[r - 1, :s]
        table[r, s:n] = perm[at:at + n - s]
        at += n - s
    assert at <= blocks
    refs = np.bincount(table[table >= 0], minlength=blocks).astype(np.int32)
    cache = rng.integers(0, 256, (layers, blocks, page, entry)).astype(np.uint8)
    return rng, cache, table, lens, refs


def check_fork(cache, table, lens, refs, parent, share, in_place=False, status=None, stream=None):
    want = fp4.fork(cache, table, lens, refs, parent, share)
    c, r = dev(cache), dev(refs)
    M, Ro = table.shape[1], len(parent)
    t_out = torch.full((Ro + 2, M + 1), 77, dtype=torch.int32, device="cuda")
    l_out = torch.full((Ro + 2,), 77, dtype=torch.int32, device="cuda")
    r_out = r if in_place else torch.full_like(r, 77)
    ws = pkg.workspace_for_cache_pages(len(lens), Ro, len(refs))
    ws.fill_(0xA5)
    args = dev(table), dev(lens), r, dev(np.asarray(parent, np.int32)), t_out[1:-1, :M], l_out[1:-1], r_out
    torch.cuda.synchronize()
    pkg.dsv4_get_device_status()
    pkg.check(pkg.dsv4_cache_fork_rows(c, *args, ws, share, stream))
    torch.cuda.synchronize()
    st = pkg.dsv4_get_device_status()
    assert st == (pkg.DSV4_ERR_BAD_INDEX if want[4] else pkg.DSV4_OK)
    assert np.array_equal(t_out[1:-1, :M].cpu(), want[1]) and np.array_equal(l_out[1:-1].cpu(), want[2])
    assert np.array_equal(r_out.cpu(), want[3]) and np.array_equal(c.cpu(), want[0])
    assert bool((t_out[0] == 77).all()) and bool((t_out[-1] == 77).all()) and bool((t_out[:, M] == 77).all())
    assert int(l_out[0]) == 77 and int(l_out[-1]) == 77
    return want


@pytest.mark.parametrize("share", [True, False])
@pytest.mark.parametrize("seed", range(8))
def test_fork_random(seed, share):
    need_gpu()
    rng, *state = pool(seed, rows=int(2 + seed), blocks=400, layers=1 + seed % 3)
    parent = rng.integers(-1, 2 + seed, 3 * seed + 1)
    check_fork(*state, parent, share, in_place=seed % 2 == 0)


@pytest.mark.parametrize("entry,page", [(400, 64), (656, 64), (400, 1), (16, 3), (48, 100)])
@pytest.mark.parametrize("share", [True, False])
def test_fork_entries_and_pages(entry, page, share):
    need_gpu()
    rng, *state = pool(31, rows=4, page=page, width=3, blocks=60, entry=entry)
    check_fork(*state, rng.integers(-1, 4, 7), share)


def test_fork_identity_frees_and_multiplies():
    need_gpu()
    _, *state = pool(32, rows=6, blocks=80)
    check_fork(*state, [0, 1, 2, 3, 4, 5], True)
    check_fork(*state, [0, -1, 2, -1, 4, -1], True, in_place=True)
    check_fork(*state, [-1] * 6, True)
    check_fork(*state, [3] * 9, True)
    check_fork(*state, [], True)
    check_fork(*state, [5], False)


def test_fork_of_many_rows():
    """More rows than threads, several tiles of pages, rows wider than a warp."""
    need_gpu()
    rng, *state = pool(33, rows=3000, page=2, width=40, blocks=150000, layers=1, fill=0.8)
    check_fork(*state, rng.integers(-1, 3000, 2500), True)
    check_fork(*state, rng.integers(-1, 3000, 1500), False)


@pytest.mark.parametrize("free", [0, 1, 2, 5, 11])
@pytest.mark.parametrize("share", [True, False])
def test_fork_without_enough_pages(free, share):
    need_gpu()
    rng, cache, table, lens, refs = pool(34, rows=6, blocks=60)
    refs = refs.copy()
    refs[np.flatnonzero(refs == 0)[free:]] = 1                     # pages that something else holds
    want = check_fork(cache, table, lens, refs, [0, 1, 1, 2, 2, 2, 3, 3, 0, 1, 4, 4, 5, 5], share, in_place=True)
    assert want[4] > 0 or share


def test_fork_bad_inputs():
    """Pages, lengths and parents out of range are flagged and left out; nothing outside the arrays is touched."""
    need_gpu()
    _, cache, table, lens, refs = pool(35, rows=4, blocks=90)
    table, lens = table.copy(), lens.copy()
    lens[:] = [20, 24, 9, 14]
    for r in range(4):
        table[r] = np.arange(6) + 6 * r
    refs = np.bincount(table.ravel(), minlength=90).astype(np.int32)
    refs[table[2, 3:]] = refs[table[3, 4:]] = 0
    table[0, 1], table[1, 2], lens[1] = 90, -5, 1000
    refs[1] = refs[8] = 0
    check_fork(cache, table, lens, refs, [0, 4, 1, 1, 2, 99, -7], True)
    check_fork(cache, table, np.array([-3, 24, 2 ** 31 - 1, -2 ** 31], np.int32), refs, [0, 1, 2, 3, 1], True)


def check_compact(cache, table, lens, refs, in_place=False):
    want = fp4.compact(cache, table, lens, refs)
    c, r, t = dev(cache), dev(refs), dev(table)
    B, M = len(refs), table.shape[1]
    guard = lambda n: torch.full((n + 2,), 77, dtype=torch.int32, device="cuda")  # noqa: E731
    r_full, m_full, l_full = guard(B), guard(B), guard(1)
    t_full = torch.full((len(lens) + 2, M + 3), 77, dtype=torch.int32, device="cuda")
    t_out, r_out = (t, r) if in_place else (t_full[1:-1, :M], r_full[1:-1])
    ws = pkg.workspace_for_cache_pages(0, 0, B)
    ws.fill_(0xA5)
    l = dev(lens)
    torch.cuda.synchronize()
    pkg.dsv4_get_device_status()
    pkg.check(pkg.dsv4_cache_compact(c, t, l, r, t_out, r_out, m_full[1:-1], l_full[1:-1], ws))
    torch.cuda.synchronize()
    st = pkg.dsv4_get_device_status()
    assert st == (pkg.DSV4_ERR_BAD_INDEX if want[5] else pkg.DSV4_OK)
    assert np.array_equal(t_out.cpu(), want[1]) and np.array_equal(r_out.cpu(), want[2])
    assert np.array_equal(m_full[1:-1].cpu(), want[3]) and int(l_full[1]) == want[4]
    assert np.array_equal(c.cpu(), want[0])
    for f in (r_full, m_full, l_full):
        assert int(f[0]) == 77 and int(f[-1]) == 77
    return want


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("seed", range(6))
def test_compact_random(seed, in_place):
    need_gpu()
    rng, cache, table, lens, refs = pool(50 + seed, rows=5, blocks=[64, 65, 127, 1000, 8192, 40][seed])
    spare = np.flatnonzero(refs == 0)
    refs[spare[rng.random(len(spare)) < 0.3]] = 3
    check_compact(cache, table, lens, refs, in_place)


@pytest.mark.parametrize("entry,page", [(400, 64), (656, 64), (400, 1), (16, 3)])
def test_compact_entries_and_pages(entry, page):
    need_gpu()
    check_compact(*pool(60, rows=4, page=page, width=4, blocks=50, entry=entry, layers=3)[1:])


def test_compact_empty_full_and_already_compact():
    need_gpu()
    _, cache, table, lens, refs = pool(61, rows=4, blocks=70)
    check_compact(cache, np.full_like(table, -1), np.zeros_like(lens), np.zeros_like(refs))
    check_compact(cache, table, lens, np.maximum(refs, 1))
    want = check_compact(cache, table, lens, refs)
    check_compact(want[0], want[1], lens, want[2], in_place=True)
    check_compact(cache, table[:0], lens[:0], refs)


def test_compact_flags_pages_without_a_count():
    need_gpu()
    _, cache, table, lens, refs = pool(62, rows=4, blocks=70)
    refs = refs.copy()
    refs[table[int(np.argmax(lens)), 0]] = 0
    refs[5] = -2 if refs[5] == 0 else refs[5]
    assert check_compact(cache, table, lens, refs)[5] > 0


def test_compact_of_a_large_pool():
    need_gpu()
    rng, cache, table, lens, refs = pool(63, rows=2000, page=2, width=30, blocks=130001, layers=1)
    check_compact(cache, table, lens, refs, in_place=True)


def check_copy(dst, src, s, d, one_pool):
    want, bad = fp4.copy_pages(dst, src, s, d, one_pool)
    dd = dev(dst)
    sd = dd if one_pool else dev(src)
    ws = pkg.workspace_for_cache_pages(0, 0, dst.shape[1])
    ws.fill_(0xA5)
    args = dev(np.asarray(s, np.int32)), dev(np.asarray(d, np.int32))
    torch.cuda.synchronize()
    pkg.dsv4_get_device_status()
    pkg.check(pkg.dsv4_cache_copy_pages(dd, sd, *args, ws))
    torch.cuda.synchronize()
    assert pkg.dsv4_get_device_status() == (pkg.DSV4_ERR_BAD_INDEX if bad else pkg.DSV4_OK)
    assert np.array_equal(dd.cpu(), want)
    if not one_pool:
        assert np.array_equal(sd.cpu(), src)


@pytest.mark.parametrize("entry,page,layers", [(400, 64, 3), (656, 16, 1), (16, 1, 5), (48, 7, 2)])
@pytest.mark.parametrize("n", [1, 2, 19])
def test_copy_two_pools(entry, page, layers, n):
    need_gpu()
    rng = np.random.default_rng(70)
    dst = rng.integers(0, 256, (layers, 40, page, entry)).astype(np.uint8)
    src = rng.integers(0, 256, (layers, 23, page, entry)).astype(np.uint8)
    check_copy(dst, src, rng.integers(0, 23, n), rng.permutation(40)[:n], False)


@pytest.mark.parametrize("page", [1, 511, 512, 513, 1024, 1025, 2048, 2049, 4100])
@pytest.mark.parametrize("n", [3, 300])
def test_copy_page_sizes(page, n):
    """Pages of 16-byte entries around the sizes where more threads share a page, or take it in several rounds."""
    need_gpu()
    rng = np.random.default_rng(page)
    dst = rng.integers(0, 256, (2, 400, page, 16)).astype(np.uint8)
    src = rng.integers(0, 256, (2, 310, page, 16)).astype(np.uint8)
    check_copy(dst, src, rng.integers(0, 310, n), rng.permutation(400)[:n], False)


def test_copy_repeats_conflicts_and_bad_pages():
    need_gpu()
    rng = np.random.default_rng(71)
    a = rng.integers(0, 256, (2, 30, 4, 32)).astype(np.uint8)
    b = rng.integers(0, 256, (2, 30, 4, 32)).astype(np.uint8)
    check_copy(a, b, [1, 2, 3, 4], [5, 5, 6, 5], False)            # the last pair of a target
    check_copy(a, a, [1, 2, 3], [5, 6, 5], True)
    check_copy(a, a, [1, 5, 7], [5, 6, 7], True)                   # 5 is a source and a target; 7 is both itself
    check_copy(a, a, [1, -1, 30, 3], [5, 6, 7, 30], True)
    check_copy(a, b, [1, -1, 30, 3], [5, 6, 7, -2], False)
    check_copy(a, a, rng.integers(-1, 31, 20000), rng.integers(-1, 31, 20000), True)
    check_copy(a, b, rng.integers(-1, 31, 20000), rng.integers(-1, 31, 20000), False)
    check_copy(a, a, [], [], True)


def test_layers_that_are_not_neighbours():
    """A pool whose layers lie apart (every second one of a larger tensor), past 32-bit offsets."""
    need_gpu()
    big = torch.zeros((4, 45000, 64, 400), dtype=torch.uint8, device="cuda")
    cache = big[::2]
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    cache[:, 44990:] = torch.randint(0, 256, (2, 10, 64, 400), dtype=torch.uint8, generator=g, device="cuda")
    want = cache[:, 44990:44993].clone()
    ws = pkg.workspace_for_cache_pages(0, 0, 45000)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    pkg.check(pkg.dsv4_cache_copy_pages(cache, cache, i32(44990, 44991, 44992), i32(7, 8, 44899), ws))
    assert torch.equal(cache[:, [7, 8, 44899]], want) and not big[1::2].any()


def test_a_run_of_them_as_a_server_makes_it():
    """Insert two prompts, fork each into three samples, append different tokens, free two samples, compact: the decode
    of the remaining rows does not change by a bit, and equals that of a cache which was never forked."""
    need_gpu()
    rng = np.random.default_rng(80)
    page, blocks, H, M, L = 16, 64, 16, 8, 2
    cache = torch.zeros((L, blocks, page, 400), dtype=torch.uint8, device="cuda")
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
    ang = rng.uniform(0, 6.28, (256, 32))
    table_cs = dev(np.concatenate([np.cos(ang), np.sin(ang)], axis=1).astype(np.float32))
    keys = {}

    def append(table, lens, what):
        """One token (or a prompt) to each row: what[r] = list of keys (bf16 bits)."""
        t, n = table.cpu().numpy(), lens.cpu().numpy()
        kv = np.concatenate([np.stack(w) for w in what if len(w)])
        pos = np.concatenate([n[r] + np.arange(len(w)) for r, w in enumerate(what)])
        slot = np.concatenate([t[r, (n[r] + np.arange(len(w))) // page] * page + (n[r] + np.arange(len(w))) % page
                               for r, w in enumerate(what) if len(w)])
        q = torch.zeros((len(kv), 1, 576), dtype=torch.bfloat16, device="cuda")
        kd = torch.from_numpy(kv.view(np.int16)).view(torch.bfloat16).cuda()
        for layer in range(L):
            pkg.check(pkg.dsv4_qk_norm_rope_kv_insert_fp4(q, q.clone(), kd, dev(pos.astype(np.int64)),
                                                          dev(slot.astype(np.int64)), table_cs, cache[layer]))
        return i32(n + [len(w) for w in what])

    def decode(table, lens, q):
        R = len(lens)
        none = torch.empty((R, 0), dtype=torch.int32, device="cuda")
        outs = [pkg.sparse_mla_decode_fp4(q, cache[layer], table, None, none, None, lens, 256, None, 0.05) for layer in range(L)]
        assert torch.equal(outs[0][0], outs[1][0])
        return outs[0]

    draw = lambda n: [synth.bf16_bits(rng.standard_normal(576)) for _ in range(n)]  # noqa: E731
    prompts = [draw(37), draw(48)]
    table = np.full((2, M), -1, np.int32)
    table[0, :3], table[1, :4] = [60, 3, 17], [9, 40, 41, 2]       # row 1 has room for its next page
    table, lens = i32(table), append(i32(table), i32([0, 0]), prompts)
    refs = torch.zeros(blocks, dtype=torch.int32, device="cuda")
    refs[[60, 3, 17, 9, 40, 41]] = 1
    table, lens, refs = pkg.cache_fork_rows(cache, table, lens, refs, i32([0, 0, 0, 1, 1, 1]))
    t = table.cpu().numpy().copy()
    fresh = np.flatnonzero(refs.cpu().numpy() == 0)[-3:]
    t[3:, 3] = fresh                                               # prompt 1 ends on a page border: a page each
    refs[torch.from_numpy(fresh).cuda()] = 1
    table = i32(t)
    tails = [draw(2) for _ in range(6)]
    lens = append(table, lens, tails)
    q = torch.randn((6, H, 576), device="cuda").bfloat16()
    out, lse = decode(table, lens, q)
    keep = [0, 2, 4, 5]
    parent = i32([r if r in keep else -1 for r in range(6)])
    table, lens, refs = pkg.cache_fork_rows(cache, table, lens, refs, parent)
    table, refs, page_map, live = pkg.cache_compact(cache, table, lens, refs)
    assert int(live) == int((refs > 0).sum()) and int(table.max()) < int(live)
    cache[:, int(live):] = 255                                     # what lies past the live pages no longer matters
    out2, lse2 = decode(table, lens, q)
    assert torch.equal(out[keep], out2[keep]) and torch.equal(lse[keep], lse2[keep])
    assert not out2[[1, 3]].any() and bool(torch.isneginf(lse2[[1, 3]]).all())
    # the same rows in a cache of their own
    cache = torch.zeros((L, blocks, page, 400), dtype=torch.uint8, device="cuda")
    t = i32(np.arange(6 * 4).reshape(6, 4))
    n = append(t, i32([0] * 6), [prompts[r // 3] + tails[r] for r in range(6)])
    out3, lse3 = decode(t, n, q)
    assert torch.equal(out, out3) and torch.equal(lse, lse3)
    torch.cuda.synchronize()
    assert pkg.dsv4_get_device_status() == pkg.DSV4_OK


def test_captured_fork_and_compact():
    need_gpu()
    rng, cache, table, lens, refs = pool(90, rows=5, blocks=100)
    parent = np.array([0, 0, 3, -1, 2, 2], np.int32)
    c0, args = dev(cache), (dev(table), dev(lens), dev(refs), dev(parent))
    c = c0.clone()
    t1, l1, r1 = pkg.cache_fork_rows(c, *args)
    t2, r2, m2, n2 = pkg.cache_compact(c, t1, l1, r1)
    cc = c0.clone()
    ws = pkg.workspace_for_cache_pages(5, 6, 100)
    outs = [torch.empty_like(x) for x in (t1, l1, r1, t2, r2, m2, n2)]
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        pkg.check(pkg.dsv4_cache_fork_rows(cc, *args, outs[0], outs[1], outs[2], ws))
        pkg.check(pkg.dsv4_cache_compact(cc, outs[0], outs[1], outs[2], outs[3], outs[4], outs[5], outs[6], ws))
    for _ in range(2):
        cc.copy_(c0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip((t1, l1, r1, t2, r2, m2, n2, c), (*outs, cc)):
            assert torch.equal(a, b)


def test_refusals():
    need_gpu()
    cache = torch.zeros((2, 8, 4, 16), dtype=torch.uint8, device="cuda")
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = pkg.workspace_for_cache_pages(3, 3, 8)
    t, l, r = i32(3, 4), i32(3), i32(8)
    fork = lambda **k: pkg.dsv4_cache_fork_rows(**{**dict(  # noqa: E731
        cache=cache, block_table=t, seq_lens=l, ref_counts=r, parent=i32(3), block_table_out=i32(3, 4),
        seq_lens_out=i32(3), ref_counts_out=r, workspace=ws), **k})
    assert fork() == pkg.DSV4_OK
    assert fork(block_table_out=t) == pkg.DSV4_ERR_INVALID_ARG
    assert fork(seq_lens_out=l) == pkg.DSV4_ERR_INVALID_ARG
    assert fork(workspace=ws[:-256]) == pkg.DSV4_ERR_INVALID_ARG
    both = i32(12)
    assert fork(ref_counts=both[:8], ref_counts_out=both[4:]) == pkg.DSV4_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        fork(ref_counts=i32(7))
    with pytest.raises(ValueError):
        fork(cache=cache.transpose(1, 2))
    with pytest.raises(TypeError):
        fork(parent=i32(3).long())
    compact = lambda **k: pkg.dsv4_cache_compact(**{**dict(  # noqa: E731
        cache=cache, block_table=t, seq_lens=l, ref_counts=r, block_table_out=t, ref_counts_out=r, page_map=i32(8),
        num_live=i32(1), workspace=ws), **k})
    assert compact() == pkg.DSV4_OK
    assert compact(page_map=r) == pkg.DSV4_ERR_INVALID_ARG
    rows = i32(4, 4)
    assert compact(block_table=rows[:3], block_table_out=rows[1:]) == pkg.DSV4_ERR_INVALID_ARG
    copy = lambda **k: pkg.dsv4_cache_copy_pages(**{**dict(  # noqa: E731
        dst_cache=cache, src_cache=cache, src_pages=i32(0), dst_pages=i32(0), workspace=ws), **k})
    assert copy() == pkg.DSV4_OK
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    assert copy(src_cache=cache[:, 2:], src_pages=one, dst_pages=one) == pkg.DSV4_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        copy(src_pages=one)
    with pytest.raises(ValueError):
        copy(src_cache=torch.zeros((1, 8, 4, 16), dtype=torch.uint8, device="cuda"))
    pkg.dsv4_get_device_status()
