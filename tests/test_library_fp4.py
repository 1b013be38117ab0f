"""CPU-only checks of the 4-bit cache's and the page operators' argument errors at the C ABI."""
import ctypes

import pytest

import sparse_mla_decode_combine_gb300 as pkg
from sparse_mla_decode_combine_gb300 import build as b

P, BAD, OK = ctypes.c_void_p(256), pkg.DSV4_ERR_INVALID_ARG, pkg.DSV4_OK


@pytest.fixture(scope="module")
def lib():
    b.build()
    return pkg.load_library()


def each(call, good, changes, want):
    for i, v in changes:
        args = list(good)
        args[i] = v
        assert call(*args) == want, (i, v)


def test_decode(lib):
    #       q, qs, kv, blocks, page, bt, bts, maxb, reqs, req, topk, ts, K, lens, seq, T, H, W, sink, scale, out, lse, ws, n, st
    good = [P, 576 * 16, P, 1, 64, P, 1, 1, 1, None, P, 4, 4, None, P, 1, 16, 8, None, 1.0, P, None, P, 0, None]
    call = lib.dsv4_sparse_mla_decode_fp4
    assert call(*good) == BAD      # no workspace
    each(call, good, [(16, 48), (16, 8), (12, 8193)], pkg.DSV4_ERR_UNSUPPORTED)
    each(call, good, [(19, float("nan")), (19, -1.0), (15, -1), (17, -1), (12, -1), (1, 9215), (1, 9216 + 4), (3, 0), (4, 0),
                      (6, 0), (8, 0), (14, None), (10, None), (11, 3), (0, None), (2, ctypes.c_void_p(8)),
                      (22, ctypes.c_void_p(16)), (4, 1 << 31 - 1)], BAD)
    each(call, good, [(15, 0)], OK)
    size = lib.dsv4_sparse_mla_decode_fp4_workspace_size
    assert size(1, 48, 4, 4) == 0 and size(1, 16, 8193, 4) == 0 and size(-1, 16, 4, 4) == 0 and size(1, 16, 4, -1) == 0


def test_insert(lib):
    #       q, qs, qo, qos, T, H, qw, kw, n, eps, kv, kvs, pos, slot, cs, maxp, cache, slots, ko, kos, st
    good = [P, 1152, P, 1152, 1, 2, None, None, 512, 1e-6, P, 576, P, P, P, 8, P, 4, ctypes.c_void_p(512), 576, None]
    call = lib.dsv4_qk_norm_rope_kv_insert_fp4
    each(call, good, [(5, 0), (5, 129), (9, float("nan")), (9, -1.0), (1, 1153), (1, 1150), (3, 1150), (11, 577), (11, 574),
                      (15, 0), (8, 64), (8, 575), (17, -1), (19, 577), (19, 100), (18, ctypes.c_void_p(2)), (0, None),
                      (10, ctypes.c_void_p(258)), (16, ctypes.c_void_p(8)), (12, None), (4, -1)], BAD)
    each(call, good, [(4, 0)], OK)
    each(call, good, [(18, P)], BAD)                       # k_out is kv
    good[4] = 2
    each(call, good, [(3, 1154), (1, 1154)], BAD)          # queries in place with another stride


def test_pages(lib):
    size = lib.dsv4_cache_pages_workspace_size
    assert size(0, 0, 0) > 0 and size(3, 5, 100) >= 20 * 100 and size(-1, 0, 4) == 0 and size(0, 0, (1 << 30) + 1) == 0
    n = size(2, 3, 8)
    at = lambda i: ctypes.c_void_p(4096 * i)  # noqa: E731
    #       cache, L, ls, B, page, entry, bt, bts, lens, R, par, Ro, M, bto, btos, lo, refs, ro, share, ws, n, st
    good = [at(100), 2, 8 * 64, 8, 4, 16, at(1), 4, at(2), 2, at(3), 3, 4, at(4), 4, at(5), at(6), at(7), 1, at(8), n - 1, None]
    fork = lib.dsv4_cache_fork_rows
    assert fork(*good) == BAD      # the workspace is a byte short
    good[20] = n
    each(fork, good, [(1, 0), (2, 8 * 64 - 16), (2, 8 * 64 + 8), (3, -1), (4, 0), (5, 24), (5, 0), (7, 3), (8, None), (10, None),
                      (12, (1 << 20) + 1), (13, at(1)), (14, 3), (15, at(2)), (16, None), (17, ctypes.c_void_p(4096 * 6 + 4)),
                      (19, None), (19, ctypes.c_void_p(16)), (0, ctypes.c_void_p(8)), (0, None)], BAD)
    #       cache, L, ls, B, page, entry, bt, bts, lens, R, M, bto, btos, refs, ro, map, live, ws, n, st
    good = [at(100), 2, 8 * 64, 8, 4, 16, at(1), 4, at(2), 2, 4, at(4), 4, at(6), at(6), at(7), at(9), at(8), n, None]
    each(lib.dsv4_cache_compact, good, [(1, 0), (5, 8), (7, 3), (8, None), (11, ctypes.c_void_p(4096 + 16)), (12, 3), (13, None),
                                        (14, ctypes.c_void_p(4096 * 6 + 8)), (15, at(6)), (15, None), (16, None), (17, None),
                                        (18, 64)], BAD)
    #       dst, dls, dB, src, sls, sB, L, page, entry, sp, dp, n, ws, wn, st
    good = [at(100), 512, 8, at(200), 512, 8, 2, 4, 16, at(1), at(2), 3, at(8), n, None]
    copy = lib.dsv4_cache_copy_pages
    each(copy, good, [(0, None), (1, 500), (3, ctypes.c_void_p(4096 * 100 + 512)), (6, 0), (8, 20), (9, None), (10, None), (11, -1),
                      (12, None), (13, 8)], BAD)
    each(copy, good, [(11, 0)], OK)
