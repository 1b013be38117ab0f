"""CPU-only: inserts whose outputs would overwrite what is still to be read are refused at the C ABI."""
import ctypes

import pytest
import torch

import sparse_mla_decode_combine_gb300 as pkg
from sparse_mla_decode_combine_gb300 import build as b

T, H, ROW, KEY = 4, 2, 2 * 2 * 576, 2 * 576      # tokens, heads, and the bytes of a token's queries and of its key
Q, QO, KV, KO = (1 << 20), (2 << 20), (3 << 20), (4 << 20)


@pytest.fixture(scope="module")
def lib():
    b.build()
    return pkg.load_library()


def call(lib, q=Q, qs=ROW, qo=QO, qos=ROW, kv=KV, kvs=KEY, ko=KO, kos=KEY, tokens=T):
    """Byte addresses and strides; nothing behind the addresses is touched by a call that is refused."""
    P = ctypes.c_void_p
    return lib.dsv4_qk_norm_rope_kv_insert_fp4(P(q), qs // 2, P(qo), qos // 2, tokens, H, None, None, 512, 1e-6, P(kv), kvs // 2,
                                               P(256), P(256), P(256), 8, P(256), 4, P(ko) if ko else None, kos // 2, None)


@pytest.mark.parametrize("change", [
    dict(ko=KV), dict(ko=KV + 4), dict(ko=KV - KEY + 4), dict(ko=KV + T * KEY - 4), dict(ko=KV + KEY),
    dict(ko=KV, kos=2 * KEY, tokens=1), dict(kvs=4 * KEY, kos=4 * KEY, ko=KV + KEY - 4), dict(kvs=4 * KEY, kos=4 * KEY, ko=KV - KEY + 4),
    dict(kvs=4 * KEY, kos=3 * KEY, ko=KV + KEY),
    dict(qo=Q + 4), dict(qo=Q + ROW), dict(qo=Q - ROW + 4), dict(qo=Q, qos=ROW + 4), dict(qo=KV), dict(qo=KV - ROW),
    dict(ko=Q), dict(ko=Q + ROW - 4), dict(ko=QO + 2 * ROW), dict(qo=Q, ko=Q + KEY)])
def test_overlaps_are_refused(lib, change):
    assert call(lib, **change) == pkg.DSV4_ERR_INVALID_ARG


def side_by_side():
    """Queries in place and keys in one buffer, k_out in another, and k_out beside the keys; rows next to each other."""
    s = ROW + KEY
    yield dict(q=Q, qs=s, qo=Q, qos=s, kv=Q + ROW, kvs=s)
    yield dict(q=Q, qs=s, qo=QO, qos=ROW, kv=Q + ROW, kvs=s)
    yield dict(q=Q, qs=s + KEY, qo=Q, qos=s + KEY, kv=Q + ROW, kvs=s + KEY, ko=Q + s, kos=s + KEY)
    yield dict(kvs=2 * KEY, kos=2 * KEY, ko=KV + KEY)
    yield dict(kvs=2 * KEY, kos=2 * KEY, ko=KV - KEY)
    yield dict(ko=KV + T * KEY)
    yield dict(ko=KV - T * KEY)
    yield dict(q=Q, qs=3 * ROW, qo=Q + ROW, qos=3 * ROW)
    yield dict(q=Q, qs=3 * ROW, qo=Q - 2 * ROW, qos=3 * ROW)
    yield dict(q=Q, qs=3 * ROW, qo=Q + 3 * ROW, qos=ROW, tokens=1)
    yield dict(ko=None)


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are made up: only a machine without a GPU takes them so far")
@pytest.mark.parametrize("change", list(side_by_side()))
def test_rows_that_do_not_meet_are_taken(lib, change):
    assert call(lib, **change) == pkg.DSV4_ERR_CUDA      # (there is no device; the arguments were taken)
