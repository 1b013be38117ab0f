"""Pins of the 4-bit oracle (oracle/fp4.py) on the CPU: the format's tables, the rounding rule by brute force, and the
page operators' invariants on small pools."""
import itertools

import numpy as np
import pytest

import oracle
from oracle import fp4


def test_e2m1_codes_round_trip_and_ties():
    assert fp4.e2m1_encode(fp4.E2M1).tolist() == list(range(8))
    assert fp4.e2m1_encode(-fp4.E2M1).tolist() == list(range(8, 16))
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    assert fp4.e2m1_encode(mids).tolist() == [0, 2, 2, 4, 4, 6, 6]
    assert fp4.e2m1_encode(np.nextafter(mids, 9)).tolist() == [1, 2, 3, 4, 5, 6, 7]
    assert fp4.e2m1_encode(np.nextafter(mids, 0)).tolist() == [0, 1, 2, 3, 4, 5, 6]
    assert fp4.e2m1_encode([100.0, np.inf, -np.inf, np.nan]).tolist() == [7, 7, 15, 7]


def test_exponent_is_the_smallest_that_fits():
    assert fp4.exponent(np.array([0.0, 6.0, np.nextafter(6.0, 7), 3.0, 1e300, 1e-60])).tolist() == [0, 0, 1, -1, 125, -127]
    for amax in np.random.default_rng(1).uniform(1e-6, 1e6, 200):
        e = int(fp4.exponent(np.array(amax)))
        assert 6.0 * 2.0 ** e >= amax > 6.0 * 2.0 ** (e - 1)


def test_entry_layout_by_hand():
    e = np.zeros((1, 400), np.uint8)
    e[0, 0] = 0x2F                     # element 0: code 15 = -6, element 1: code 2 = 1
    e[0, 255] = 0x90                   # element 511: code 9 = -1/2
    e[0, 384:400] = 127
    e[0, 384], e[0, 399] = 130, 120    # block 0 x 8, block 15 x 2^-7
    e[0, 256:258] = [0x80, 0x3F]       # BF16 1.0
    k = fp4.dequant(e)[0]
    assert (k[0], k[1], k[511], k[512]) == (-48.0, 8.0, -0.5 / 128, 1.0) and np.count_nonzero(k) == 4


def test_pack_then_dequant_is_within_half_a_step():
    x = np.random.default_rng(2).standard_normal((50, 512)) * np.ldexp(1.0, np.arange(50) - 25)[:, None]
    k = fp4.dequant(fp4.pack(x, np.zeros((50, 64), np.uint16)))[:, :512]
    amax = np.repeat(np.abs(x).reshape(50, 16, 32).max(-1), 32, axis=1)
    assert np.all(np.abs(k - x) <= amax / 6 * 1.0 * 2)   # the largest step is 2 in a block scaled to at most 6: half is 1
    assert np.array_equal(fp4.dequant(fp4.pack(k, np.zeros((50, 64), np.uint16)))[:, :512], k)


def test_bf16_rounding_matches_the_oracle_library():
    bits = np.random.default_rng(3).integers(0, 0x7F80, 500).astype(np.uint16)
    x = fp4.bf16_to_f64(bits)
    assert np.array_equal(x, [oracle.bf16_to_f64(int(b)) for b in bits])
    assert np.array_equal(fp4.f64_to_bf16(x), bits)


def pool(rng, rows, page=4, width=6, blocks=40, layers=2):
    """Rows with private pages, the first two sharing their full ones."""
    perm, at = rng.permutation(blocks), 0
    table, lens = np.full((rows, width), -1, np.int32), rng.integers(0, width * page + 1, rows).astype(np.int32)
    for r in range(rows):
        n = -(-int(lens[r]) // page)
        table[r, :n] = perm[at:at + n]
        at += n
    if rows > 1:
        s = min(lens[0], lens[1]) // page
        table[1, :s] = table[0, :s]
    refs = np.bincount(table[table >= 0], minlength=blocks).astype(np.int32)
    return rng.integers(0, 256, (layers, blocks, page, 16)).astype(np.uint8), table, lens, refs


def row_bytes(cache, table, lens, r):
    page = cache.shape[2]
    n = -(-int(lens[r]) // page)
    return cache[:, table[r, :n]].reshape(cache.shape[0], -1, cache.shape[3])[:, :lens[r]]


@pytest.mark.parametrize("seed,share", list(itertools.product(range(6), (True, False))))
def test_fork_keeps_every_row_and_counts_every_reference(seed, share):
    rng = np.random.default_rng(seed)
    cache, table, lens, refs = pool(rng, 4, blocks=120)
    parent = rng.integers(-1, 4, 6).astype(np.int32)
    c, t, n, r, bad = fp4.fork(cache, table, lens, refs, parent, share)
    assert bad == 0
    for i, par in enumerate(parent):
        assert n[i] == (lens[par] if par >= 0 else 0)
        if par >= 0:
            assert np.array_equal(row_bytes(c, t, n, i), row_bytes(cache, table, lens, par))
    assert np.array_equal(r, np.bincount(t[t >= 0], minlength=len(refs)))
    page = cache.shape[2]
    for i in range(len(parent)):       # a partly filled page has one holder; without sharing every page has
        for j in range(-(-int(n[i]) // page)):
            if not share or (j + 1) * page > n[i]:
                assert r[t[i, j]] == 1


@pytest.mark.parametrize("seed", range(6))
def test_compact_keeps_every_row(seed):
    rng = np.random.default_rng(seed)
    cache, table, lens, refs = pool(rng, 4, blocks=60)
    refs[np.flatnonzero(refs == 0)[:3]] = 2
    c, t, r, to, live, bad = fp4.compact(cache, table, lens, refs)
    assert bad == 0 and live == (refs > 0).sum() and np.all(r[:live] > 0) and np.all(r[live:] == 0)
    for i in range(4):
        assert np.array_equal(row_bytes(c, t, lens, i), row_bytes(cache, table, lens, i))
    for b in np.flatnonzero(refs):
        assert r[to[b]] == refs[b] and np.array_equal(c[:, to[b]], cache[:, b])
