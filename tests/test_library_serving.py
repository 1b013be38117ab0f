"""CPU-only checks of the argument errors of draft verification, key weights and eviction at the C ABI."""
import ctypes

import pytest

import sparse_mla_decode_combine_gb300 as pkg
from sparse_mla_decode_combine_gb300 import build as b

P, BAD, OK = ctypes.c_void_p(256), pkg.DSV4_ERR_INVALID_ARG, pkg.DSV4_OK
at = lambda i: ctypes.c_void_p(65536 * i)  # noqa: E731


@pytest.fixture(scope="module")
def lib():
    b.build()
    return pkg.load_library()


def each(call, good, changes, want):
    for i, v in changes:
        args = list(good)
        args[i] = v
        assert call(*args) == want, (i, v)


def test_verify(lib):
    #       p, ps, q, qs, bf16, V, tok, Nd, start, R, N, u, greedy, out, os, ow, acc, seq, seqo, st
    good = [P, 100, P, 100, 0, 100, P, 3, P, 2, 5, P, None, P, 4, 4, P, None, None, None]
    call = lib.dsv4_verify_drafts
    each(call, good, [(0, None), (1, 99), (3, 99), (5, 0), (5, (1 << 22) + 1), (6, None), (7, -1), (8, None), (9, -1),
                      (9, (1 << 24) + 1), (10, -1), (11, None), (13, None), (14, 3), (15, 0), (16, None), (17, P), (18, P),
                      (0, ctypes.c_void_p(258)), (2, ctypes.c_void_p(258))], BAD)
    each(call, good, [(9, 0)], OK)
    good[4] = 1
    each(call, good, [(0, ctypes.c_void_p(257)), (2, ctypes.c_void_p(257))], BAD)


def test_key_weights(lib):
    size = lib.dsv4_sparse_mla_key_weights_workspace_size
    assert size(1, 48, 4, 4) == 0 and size(1, 16, 8193, 4) == 0 and size(-1, 16, 4, 4) == 0 and size(1, 16, 4, -1) == 0
    assert size(1, 16, 4, (1 << 24) + 1) == 0
    n = size(3, 16, 4, 8)
    assert n >= 3 * 12 * 4 * 2
    #       q, qs, kv, blocks, page, entry, bt, bts, maxb, reqs, req, topk, ts, K, lens, seq, T, H, W, lse, scale, w, wst, ww, ws, n, st
    good = [P, 576 * 16, P, 1, 64, 400, P, 1, 1, 3, None, P, 4, 4, None, P, 3, 16, 8, P, 1.0, P, 64, 64, P, n, None]
    call = lib.dsv4_sparse_mla_key_weights
    each(call, good, [(17, 48), (17, 8), (13, 8193), (5, 576), (5, 0)], pkg.DSV4_ERR_UNSUPPORTED)
    each(call, good, [(20, float("nan")), (20, -1.0), (16, -1), (18, -1), (13, -1), (1, 9215), (1, 9216 + 4), (4, 0), (3, -1),
                      (7, 0), (8, 0), (9, 0), (9, 2), (15, None), (11, None), (12, 3), (0, None), (19, None), (21, None), (22, 63),
                      (23, 63), (24, None), (24, ctypes.c_void_p(128)), (25, n - 1), (2, ctypes.c_void_p(8)), (2, None),
                      (6, None), (3, 1 << 26), (0, ctypes.c_void_p(264)), (21, ctypes.c_void_p(258))], BAD)
    each(call, good, [(16, 0)], OK)


def test_evict(lib):
    size = lib.dsv4_cache_evict_workspace_size
    n = size(2, 4, 8, 2, 4, 16, 6)
    assert n > 0
    for bad in [(-1, 4, 8, 2, 4, 16, 6), (2, -1, 8, 2, 4, 16, 6), (2, 4, -1, 2, 4, 16, 6), (2, 4, 8, 0, 4, 16, 6),
                (2, 4, 8, 2, 0, 16, 6), (2, 4, 8, 2, 4, 24, 6), (2, 4, 8, 2, 4, 16, 0), (2, (1 << 20) + 1, 8, 2, 1, 16, 6),
                (2, 4, (1 << 30) + 1, 2, 4, 16, 6), (2, 1 << 20, 8, 2, 1 << 12, 16, 6), (1 << 30, 4, 8, 64, 4, 16, 6)]:
        assert size(*bad) == 0, bad
    #       cache, L, ls, B, page, entry, bt, bts, lens, R, M, w, wst, ww, budget, limit, first, recent, bto, btos, lo, refs,
    #       ro, wo, wos, ws, n, st
    good = [at(100), 2, 8 * 64, 8, 4, 16, at(1), 4, at(2), 2, 4, at(3), 16, 16, 6, 7, 2, 2, at(4), 4, at(5), at(6), at(7), at(8),
            16, at(9), n, None]
    call = lib.dsv4_cache_evict
    each(call, good, [(26, n - 1), (25, None), (25, ctypes.c_void_p(65536 * 9 + 128)), (0, None), (0, ctypes.c_void_p(8)), (1, 0),
                      (2, 8 * 64 - 16), (2, 8 * 64 + 8), (4, 0), (5, 8), (6, None), (7, 3), (8, None), (9, -1), (10, -1), (11, None),
                      (12, 15), (13, 15), (14, 0), (15, 5), (16, -1), (17, -1), (16, 5), (17, 5), (18, None), (19, 3), (20, None),
                      (21, None), (22, None), (23, None), (24, 15)], BAD)
    # rows that are read while others are written
    each(call, good, [(18, at(1)), (18, ctypes.c_void_p(65536 + 16)), (20, at(2)), (22, ctypes.c_void_p(65536 * 6 + 4)),
                      (23, ctypes.c_void_p(65536 * 3 + 64))], BAD)
    same = list(good)
    same[23], same[24] = at(3), 17
    assert call(*same) == BAD      # weights in place with another stride
    none = list(good)
    none[9], none[21] = 0, at(7)
    assert call(*none) == OK
