"""CPU-only: calls whose outputs share bytes with what is still read are refused at the C ABI."""
import ctypes

import pytest
import torch

import sparse_mla_decode_combine_gb300 as pkg
from sparse_mla_decode_combine_gb300 import build as b

BAD = pkg.DSV4_ERR_INVALID_ARG
made_up = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are made up: only a machine without a GPU takes them so far")
MB = 1 << 20
R, V, N, W = 4, 100, 12, 6                   # requests, vocabulary, rows, width of the tokens
VERIFY = dict(target=MB, draft=2 * MB, tokens=3 * MB, start=4 * MB, uniform=5 * MB, greedy=6 * MB, out=7 * MB, accepted=8 * MB,
              seq=9 * MB, seq_out=9 * MB)


@pytest.fixture(scope="module")
def lib():
    b.build()
    return pkg.load_library()


def P(x):
    return ctypes.c_void_p(x)


def verify(lib, stride=W, **change):
    """Byte addresses; nothing behind them is touched by a call that is refused."""
    a = {**VERIFY, **change}
    return lib.dsv4_verify_drafts(P(a["target"]), V, P(a["draft"]), V, 0, V, P(a["tokens"]), N - R, P(a["start"]), R, N,
                                  P(a["uniform"]), P(a["greedy"]), P(a["out"]), stride, W, P(a["accepted"]), P(a["seq"]),
                                  P(a["seq_out"]), None)


# the inputs' sizes in bytes
INPUTS = dict(target=4 * N * V, draft=4 * (N - R) * V, tokens=4 * (N - R), start=4 * (R + 1), uniform=4 * N, greedy=R, seq=4 * R)


@pytest.mark.parametrize("name", INPUTS)
def test_verify(lib, name):
    at, n = VERIFY[name], INPUTS[name]
    for out, size in (("out", 4 * R * W), ("accepted", 4 * R)):
        for shift in (0, n // 4 * 4 - 4 if n > 4 else 0, 4 - size):
            assert verify(lib, **{out: at + shift}) == BAD, (out, shift)
    if name != "seq":
        assert verify(lib, seq_out=at) == BAD
    else:
        assert verify(lib, seq_out=at + 4) == BAD and verify(lib, seq_out=at - 4) == BAD


def test_verify_outputs_among_themselves(lib):
    for a, b_ in (("out", "accepted"), ("out", "seq_out"), ("accepted", "seq_out"), ("accepted", "seq")):
        assert verify(lib, **{a: VERIFY[b_]}) == BAD, (a, b_)
    assert verify(lib, stride=10, accepted=VERIFY["out"] + 4 * (3 * 10 + W - 1)) == BAD


@made_up
def test_verify_arrays_that_do_not_meet_are_taken(lib):
    gap = VERIFY["out"] + 4 * W             # between two rows of `out`, which are 10 values apart
    for change in (dict(), dict(seq_out=10 * MB), dict(seq=None, seq_out=None), dict(stride=10, accepted=gap), dict(stride=10, seq_out=gap),
                   dict(out=VERIFY["tokens"] - 4 * R * W), dict(out=VERIFY["tokens"] + 4 * (N - R)), dict(draft=None)):
        assert verify(lib, **change) == pkg.DSV4_ERR_CUDA, change       # (there is no device; the arguments were taken)


WEIGHTS = dict(q=MB, kv=2 * MB, table=3 * MB, req=4 * MB, topk=5 * MB, lens=6 * MB, seq=7 * MB, lse=8 * MB, weights=9 * MB, ws=10 * MB)
T, H = 5, 16                                 # rows of 2 pages of 64 entries; 3 rows
WEIGHTS_INPUTS = dict(q=2 * T * H * 576, kv=7 * 64 * 400, table=4 * 3 * 2, req=4 * T, topk=4 * T * 8, lens=4 * T, seq=4 * T, lse=4 * T * H)


def key_weights(lib, stride=128, **change):
    a = {**WEIGHTS, **change}
    n = lib.dsv4_sparse_mla_key_weights_workspace_size(T, H, 8, 4)
    return lib.dsv4_sparse_mla_key_weights(P(a["q"]), 576 * H, P(a["kv"]), 7, 64, 400, P(a["table"]), 2, 2, 3, P(a["req"]), P(a["topk"]), 8,
                                           8, P(a["lens"]), P(a["seq"]), T, H, 4, P(a["lse"]), 1.0, P(a["weights"]), stride, 128,
                                           P(a["ws"]), n, None)


@pytest.mark.parametrize("name", WEIGHTS_INPUTS)
def test_key_weights(lib, name):
    at, n = WEIGHTS[name], WEIGHTS_INPUTS[name]
    for first in (at, at + n - 4, at + 4 - 4 * 3 * 128):
        assert key_weights(lib, weights=first) == BAD, first
    for first in (at, at + (n - 1) // 256 * 256):
        assert key_weights(lib, ws=first) == BAD, first


def test_key_weights_table_over_the_workspace(lib):
    assert key_weights(lib, weights=WEIGHTS["ws"]) == BAD and key_weights(lib, weights=WEIGHTS["ws"] - 4 * 3 * 128 + 4) == BAD


@made_up
def test_key_weights_arrays_that_do_not_meet_are_taken(lib):
    gap = WEIGHTS["weights"] + 4 * 128       # between two rows of a table whose rows are 256 values apart
    for change in (dict(), dict(lens=None), dict(stride=256, lse=gap), dict(stride=256, seq=gap), dict(weights=WEIGHTS["seq"] + 4 * T),
                   dict(weights=WEIGHTS["seq"] - 4 * 3 * 128)):
        assert key_weights(lib, **change) == pkg.DSV4_ERR_CUDA, change


EVICT = dict(table=MB, lens=2 * MB, weights=3 * MB, table_out=4 * MB, lens_out=5 * MB, refs=6 * MB, refs_out=7 * MB, left=8 * MB, ws=9 * MB)
E_R, E_M, E_B = 3, 4, 9                      # rows of 4 pages of 4 entries; 9 pages
EVICT_SIZES = dict(table=4 * E_R * E_M, lens=4 * E_R, refs=4 * E_B, weights=4 * E_R * 16, table_out=4 * E_R * E_M, lens_out=4 * E_R,
                   refs_out=4 * E_B, left=4 * E_R * 16)


def evict(lib, stride=16, **change):
    a = {**EVICT, **change}
    n = lib.dsv4_cache_evict_workspace_size(E_R, E_M, E_B, 2, 4, 16, 6)
    return lib.dsv4_cache_evict(P(64 * MB), 2, 16 * 4 * E_B, E_B, 4, 16, P(a["table"]), E_M, P(a["lens"]), E_R, E_M, P(a["weights"]),
                                stride, 16, 6, 7, 2, 2, P(a["table_out"]), E_M, P(a["lens_out"]), P(a["refs"]), P(a["refs_out"]),
                                P(a["left"]), stride, P(a["ws"]), n, None)


@pytest.mark.parametrize("out", ["table_out", "lens_out", "refs_out", "left"])
def test_evict(lib, out):
    pairs = {("refs_out", "refs"), ("left", "weights")}
    for name, n in EVICT_SIZES.items():
        if name != out:
            for shift in (0, n - 4, 4 - EVICT_SIZES[out]):
                if shift or (out, name) not in pairs:
                    assert evict(lib, **{out: EVICT[name] + shift}) == BAD, (name, shift)
    assert evict(lib, **{out: EVICT["ws"]}) == BAD


def test_evict_workspace(lib):
    for name in ("table", "lens", "refs", "weights"):
        assert evict(lib, ws=EVICT[name]) == BAD, name


@made_up
def test_evict_arrays_that_do_not_meet_are_taken(lib):
    gap = EVICT["left"] + 4 * 16             # between two rows of weights that are 64 values apart
    for change in (dict(), dict(refs_out=EVICT["refs"]), dict(left=EVICT["weights"]), dict(stride=64, lens_out=gap),
                   dict(stride=64, table_out=gap), dict(stride=64, left=EVICT["weights"] + 4 * 16), dict(lens_out=EVICT["lens"] + 4 * E_R)):
        assert evict(lib, **change) == pkg.DSV4_ERR_CUDA, change
