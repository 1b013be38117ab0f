"""dsv4_qk_norm_rope_kv_insert_fp4 on the GPU against the fp64 oracle.

The entries' codes and scale bytes must match bit for bit (they are those of the exact key).  A query value, and a rope
value of the key, is computed in fp32 (at most 16 roundings of 2^-24 on the value or, for a rotated one, on its pair's
norm: 2^-20) and rounded once to BF16 (half a step, 2^-8 of the value)."""
import numpy as np
import pytest
import torch

import sparse_mla_decode_combine_gb300 as pkg
import synth
from gpu_util import need_gpu
from oracle import fp4

pytestmark = pytest.mark.gpu


def table_of(rng, max_pos):
    ang = rng.uniform(0, 2 * np.pi, (max_pos, 32))
    return np.concatenate([np.cos(ang), np.sin(ang)], axis=1).astype(np.float32)


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).view(torch.bfloat16).cuda()


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def near(got_bits, want, what):
    """BF16 bits [..., 576] against fp64 values: latent and rotated part."""
    g = fp4.bf16_to_f64(got_bits)
    pair = np.sqrt(want[..., 512::2] ** 2 + want[..., 513::2] ** 2)
    slack = np.concatenate([np.abs(want[..., :512]), np.repeat(pair, 2, axis=-1)], axis=-1) * 2.0 ** -20
    bad = ~(np.abs(g - want) <= 2.0 ** -8 * np.abs(want) + slack + 2.0 ** -133)
    assert not bad.any(), (what, np.argwhere(bad)[:3])


def run_case(seed, T, H, norm_dims=512, weights=True, in_place=False, bad=True, eps=1e-6, gap=0, k_out=True, kv=None,
             num_slots=300, max_pos=512, stream=None):
    rng = np.random.default_rng(seed)
    q = synth.bf16_bits(rng.standard_normal((T, H, 576)) * rng.uniform(0.01, 30, (T, H, 1)))
    if kv is None:
        kv = synth.bf16_bits(rng.standard_normal((T, 576)) * np.ldexp(1.0, rng.integers(-20, 20, (T, 1))))
    pos = rng.integers(0, max_pos, T)
    slots = rng.permutation(max(num_slots, T))[:T]
    num_slots = max(num_slots, T)
    if bad and T >= 5:
        slots[0], slots[1], pos[2], pos[3] = -1, num_slots + 3, max_pos, -1
    q_w = rng.uniform(0.5, 1.5, 576).astype(np.float32) if weights else None
    kv_w = rng.uniform(0.5, 1.5, norm_dims).astype(np.float32) if weights and norm_dims else None
    table = table_of(rng, max_pos)
    cache0 = rng.integers(0, 256, (num_slots, 400)).astype(np.uint8)
    want_q, want_k, want_cache, bads = fp4.insert(q, kv, pos, slots, table, cache0, q_w, kv_w, norm_dims, eps)

    wide = torch.zeros((T, H * 576 + gap), dtype=torch.bfloat16, device="cuda")
    qd = wide[:, :H * 576].view(T, H, 576)
    qd.copy_(bf16(q))
    q_out = qd if in_place else torch.empty((T, H, 576), dtype=torch.bfloat16, device="cuda")
    kd = torch.full((T + 2, 576 + gap), -3.0, dtype=torch.bfloat16, device="cuda")
    ko = kd[1:-1, :576] if k_out else None
    dev = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    cache = dev(cache0.copy())
    args = (bf16(kv), dev(pos.astype(np.int64)), dev(slots.astype(np.int64)), dev(table), cache, ko, dev(q_w), dev(kv_w))
    torch.cuda.synchronize()
    pkg.dsv4_get_device_status()
    pkg.check(pkg.dsv4_qk_norm_rope_kv_insert_fp4(qd, q_out, *args, norm_dims, eps, stream))
    torch.cuda.synchronize()
    assert (pkg.dsv4_get_device_status() == pkg.DSV4_ERR_BAD_INDEX) == (bads > 0)
    near(bits(q_out), want_q, "q")
    got = cache.cpu().numpy()
    same = np.r_[0:256, 384:400]
    assert np.array_equal(got[:, same], want_cache[:, same]), np.argwhere(got[:, same] != want_cache[:, same])[:4]
    wrote = [t for t in range(T) if 0 <= slots[t] < num_slots and 0 <= pos[t] < max_pos]
    rest = np.setdiff1d(np.arange(num_slots), slots[wrote])
    assert np.array_equal(got[rest], cache0[rest])
    held = fp4.dequant(fp4.pack(want_k[:, :512], np.zeros((T, 64), np.uint16)))[:, :512]
    rope = np.ascontiguousarray(got[slots[wrote], 256:384]).view("<u2")
    want = np.concatenate([held, want_k[:, 512:]], axis=1)
    near(np.concatenate([fp4.f64_to_bf16(held[wrote]), rope], axis=1), want[wrote], "rope")
    if k_out:
        kb = bits(ko)
        assert np.array_equal(fp4.bf16_to_f64(kb[:, :512]), fp4.bf16_to_f64(fp4.f64_to_bf16(held)))
        near(kb, np.concatenate([fp4.bf16_to_f64(kb[:, :512]), want_k[:, 512:]], axis=1), "k_out")
        assert np.array_equal(kb[wrote, 512:], rope)
        assert bool((kd[0] == -3).all()) and bool((kd[-1] == -3).all()) and (gap == 0 or bool((kd[:, 576:] == -3).all()))


@pytest.mark.parametrize("H", [1, 2, 3, 16, 17, 64, 127, 128])
def test_heads(H):
    need_gpu()
    run_case(100 + H, T=37, H=H)


@pytest.mark.parametrize("norm_dims", [0, 512, 576])
@pytest.mark.parametrize("weights", [False, True])
def test_norms(norm_dims, weights):
    need_gpu()
    run_case(200 + norm_dims, T=301, H=4, norm_dims=norm_dims, weights=weights, gap=8)


@pytest.mark.parametrize("T", [1, 2, 151, 153, 700])
def test_tokens(T):
    need_gpu()
    run_case(300 + T, T=T, H=16, bad=T > 100)


def test_in_place_odd_strides_no_k_out():
    need_gpu()
    run_case(400, T=20, H=8, in_place=True, gap=2, k_out=False)


def test_many_tokens_are_exact():
    """Four million latent values: a quantisation in fp32 alone puts about a dozen on the wrong side of a border."""
    need_gpu()
    run_case(401, T=8000, H=1, weights=True, bad=False)


def test_ties_and_block_maxima_on_the_border():
    """Without a norm the key is BF16 and ties are exact: nearest even, and a maximum of exactly 6 * 2^e keeps e."""
    need_gpu()
    rng = np.random.default_rng(402)
    x = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -1.25, -5.0, -6.0, 0.0, -0.0], (64, 576))
    x *= np.ldexp(1.0, rng.integers(-30, 30, (64, 1)))
    run_case(403, T=64, H=1, norm_dims=0, weights=False, bad=False, kv=synth.bf16_bits(x))


def test_normalised_ties():
    """Rows of one magnitude m normalise to exactly +-1 with eps 0; weights put values on borders."""
    need_gpu()
    rng = np.random.default_rng(404)
    T = 32
    x = np.where(rng.random((T, 576)) < 0.5, -1.0, 1.0) * np.ldexp(1.0, rng.integers(-8, 8, (T, 1)))
    w = rng.choice([0.25, 0.75, 1.25, 2.5, 5.0, 6.0, 0.0], 512).astype(np.float32)
    q = torch.ones((T, 1, 576), dtype=torch.bfloat16, device="cuda")
    cache = torch.zeros((T, 400), dtype=torch.uint8, device="cuda")
    table = np.concatenate([np.ones((4, 32)), np.zeros((4, 32))], axis=1).astype(np.float32)
    kv = synth.bf16_bits(x)
    pkg.check(pkg.dsv4_qk_norm_rope_kv_insert_fp4(
        q, torch.empty_like(q), bf16(kv), torch.zeros(T, dtype=torch.int64, device="cuda"),
        torch.arange(T, device="cuda"), torch.from_numpy(table).cuda(), cache, None, None, torch.from_numpy(w).cuda(), 512,
        0.0))
    want = fp4.insert(np.full((T, 1, 576), 0x3F80, np.uint16), kv, np.zeros(T, int), np.arange(T), table,
                      np.zeros((T, 400), np.uint8), None, w, 512, 0.0)[2]
    got = cache.cpu().numpy()
    assert np.array_equal(got[:, np.r_[0:256, 384:400]], want[:, np.r_[0:256, 384:400]])


@pytest.mark.parametrize("norm_dims", [0, 512])
def test_extreme_magnitudes(norm_dims):
    """All zero keys, the smallest and largest BF16 values, infinities and NaN."""
    need_gpu()
    x = np.zeros((8, 576), np.uint16)
    x[1] = 1                                   # the smallest subnormal
    x[2, :512] = 0x7F7F                        # the largest finite value (a rotated pair of it would overflow)
    x[3, ::7] = 0x0080                         # the smallest normal, among zeros
    x[4, 5], x[4, 40] = 0x7F80, 0xFF80         # infinities
    x[5, 9] = 0x7FC0                           # NaN
    x[6, :512] = np.where(np.arange(512) % 2, 0x3F80, 0x0001)
    x[7] = 0x8000                              # minus zero
    rows = slice(0, 8) if norm_dims == 0 else np.r_[0:2, 3, 6, 7]   # the square of the largest value overflows nothing in fp64
    run_case(405, T=len(x[rows]), H=1, norm_dims=norm_dims, weights=False, bad=False, kv=x[rows], eps=1e-30)


def test_insert_then_decode_reads_the_entries():
    """The decode over freshly inserted entries returns k_out's latent."""
    need_gpu()
    rng = np.random.default_rng(406)
    T = 5
    cache = torch.zeros((1, 64, 400), dtype=torch.uint8, device="cuda")
    q = torch.zeros((T, 16, 576), dtype=torch.bfloat16, device="cuda")
    k = torch.empty((T, 576), dtype=torch.bfloat16, device="cuda")
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    pkg.check(pkg.dsv4_qk_norm_rope_kv_insert_fp4(q, q, bf16(synth.bf16_bits(rng.standard_normal((T, 576)))),
                                                  dev(np.arange(T)), dev(np.arange(T)), dev(table_of(rng, 8)), cache, k))
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    out, lse = pkg.sparse_mla_decode_fp4(q, cache, i32(0).view(1, 1), i32(*[0] * T), torch.empty((T, 0), dtype=torch.int32, device="cuda"),
                                         None, i32(*range(1, T + 1)), 1, None, 1.0)
    assert torch.equal(out, k[:, None, :512].expand(T, 16, 512)) and not lse.any()


def test_captured():
    need_gpu()
    rng = np.random.default_rng(407)
    T, H = 6, 4
    q = bf16(synth.bf16_bits(rng.standard_normal((T, H, 576))))
    kv = bf16(synth.bf16_bits(rng.standard_normal((T, 576))))
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    pos, slots, table = dev(np.arange(T)), dev(np.arange(T)), dev(table_of(rng, 16))
    a, b = (torch.zeros((8, 400), dtype=torch.uint8, device="cuda") for _ in range(2))
    qa, qb = torch.empty_like(q), torch.empty_like(q)
    pkg.check(pkg.dsv4_qk_norm_rope_kv_insert_fp4(q, qa, kv, pos, slots, table, a))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkg.check(pkg.dsv4_qk_norm_rope_kv_insert_fp4(q, qb, kv, pos, slots, table, b))
    for _ in range(2):
        b.zero_()
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(qa, qb)


def test_refusals():
    need_gpu()
    q = torch.zeros((2, 2, 576), dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros((2, 576), dtype=torch.bfloat16, device="cuda")
    i = torch.zeros(2, dtype=torch.int64, device="cuda")
    table = torch.zeros((4, 64), device="cuda")
    cache = torch.zeros((4, 400), dtype=torch.uint8, device="cuda")
    call = lambda **k: pkg.dsv4_qk_norm_rope_kv_insert_fp4(**{**dict(  # noqa: E731
        q=q, q_out=q, kv=kv, positions=i, slot_mapping=i, cos_sin_cache=table, kv_cache=cache), **k})
    assert call(kv_norm_dims=64) == pkg.DSV4_ERR_INVALID_ARG
    assert call(eps=-1.0) == pkg.DSV4_ERR_INVALID_ARG
    assert call(eps=float("nan")) == pkg.DSV4_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        call(kv_norm_weight=torch.ones(576, device="cuda"))
    with pytest.raises(ValueError):
        call(q_out=q[:1])
    with pytest.raises(ValueError):
        call(positions=i[:1])
    with pytest.raises(ValueError):
        call(kv_cache=torch.zeros((4, 656), dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError):
        call(slot_mapping=i.int())
    with pytest.raises(ValueError):
        call(k_out=kv[:, :512])
    assert call(k_out=kv) == pkg.DSV4_ERR_INVALID_ARG
    wide = torch.zeros((2, 3, 576), dtype=torch.bfloat16, device="cuda")[:, :2]
    flat = torch.as_strided(wide, (2, 2, 576), (1152, 576, 1))
    assert call(q=wide, q_out=flat) == pkg.DSV4_ERR_INVALID_ARG   # in place, but rows in other places
    assert call(q=wide, q_out=wide) == pkg.DSV4_OK
    assert pkg.dsv4_get_device_status() == pkg.DSV4_OK
