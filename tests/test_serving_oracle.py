"""The oracle of draft verification, key weights and eviction, pinned by cases worked out by hand."""
import numpy as np

import synth
from oracle import fp4, serving


def test_drawn_is_the_first_sum_above():
    w = np.array([0.0, 0.25, 0.0, 0.5, 0.25, 0.0])
    assert [serving.drawn(w, u)[0] for u in (0.0, 0.24, 0.25, 0.5, 0.74, 0.75, 0.999, 1.0)] == [1, 1, 3, 3, 3, 4, 4, 4]


def test_verify_by_hand():
    p = np.array([[0.5, 0.5, 0.0], [0.25, 0.25, 0.5], [0.0, 0.0, 1.0], [0.2, 0.3, 0.5]])
    q = np.array([[1.0, 0.0, 0.0], [0.0, 1.0, 0.0]])
    # request 0: draft 0 stands (0.4 * 1 < 0.5), draft 1 does not (0.25 * 1 < 0.25 fails); what is left of row 1 is
    # (0.25, 0, 0.5): 0.3 of it is 0.225, below 0.25.  Request 1 has no draft: 0.5 of (0.2, 0.3, 0.5) lies on a border
    out, acc, seq, may, bad = serving.verify(p, q, [0, 1], [0, 3, 4], [0.4, 0.25, 0.3, 0.5], seq=[10, 4])
    assert out.tolist() == [[0, 0, -1], [2, -1, -1]] and acc.tolist() == [1, 0] and seq.tolist() == [9, 4] and bad == 0
    # without draft probabilities the drafted token has all: row 1 leaves (0.25, 0, 0.5) as well
    assert serving.verify(p, None, [0, 1], [0, 3, 4], [0.4, 0.25, 0.3, 0.2])[0].tolist() == [[0, 0, -1], [1, -1, -1]]
    # greedy: the lowest of equal ones
    out, acc, _, _, _ = serving.verify(p, None, [0, 2], [0, 3, 4], [0] * 4, greedy=[1, 1])
    assert out.tolist() == [[0, 2, 2], [2, -1, -1]] and acc.tolist() == [2, 0]
    assert serving.largest([np.nan, -np.inf, -np.inf]) == 1 and serving.largest([np.nan]) == -1


def test_verify_leaves_the_target_distribution():
    rng = np.random.default_rng(1)
    p, q = np.array([0.5, 0.2, 0.2, 0.1]), np.array([0.1, 0.5, 0.2, 0.2])
    n, seen = 20000, np.zeros(4)
    for _ in range(n):
        d = rng.choice(4, p=q)
        seen[serving.verify(np.stack([p, p]), q[None], [d], [0, 2], rng.random(2))[0][0, 0]] += 1
    # a count of n draws is off by more than 5 standard deviations once in a million times
    assert np.all(np.abs(seen - n * p) < 5 * np.sqrt(n * p * (1 - p)))


def test_key_weights_sum_to_what_the_keys_have_of_the_softmax():
    w = synth.make_workload(name="w", seed=3, heads=16, req_seq_lens=[40, 9, 0], topk_width=12, window=8, sink=False)
    import oracle
    _, lse, _ = oracle.sparse_mla_decode(w)
    got, _, adds, bad = serving.key_weights(w, lse, np.zeros((3, w.block_table.shape[1] * w.page)))
    assert np.allclose(got.sum(1), [16, 16, 0], rtol=1e-9) and bad == 0 and adds.max() == 1
    assert np.allclose(serving.dequant8(w.kv_cache.reshape(-1, 656)[:50])[:, 512:],
                       fp4.bf16_to_f64(w.kv_cache.reshape(-1, 656)[:50, 512:640].copy().view("<u2")))


def test_evict_by_hand():
    cache = np.arange(6, dtype=np.uint8)[None, :, None, None] * 2 + np.arange(2, dtype=np.uint8)[None, None, :, None]
    table, lens = np.array([[0, 1, 2], [0, 4, -1]], np.int32), np.array([6, 3], np.int32)
    refs = np.array([2, 1, 1, 0, 1, 0], np.int32)
    weights = np.array([[9, 1, 5, 1, 7, 0], [1, 2, 3, 0, 0, 0]], np.float32)
    c, t, n, r, wt, bad = serving.evict(cache, table, lens, refs, weights, 4, 4, 1, 1)
    # row 0 keeps 0, 2, 4, 5: its page 0 is shared, so page 3 takes its place; page 1 is written in place, page 2 is free
    assert t.tolist() == [[3, 1, -1], [0, 4, -1]] and n.tolist() == [4, 3] and r.tolist() == [1, 1, 0, 1, 1, 0] and bad == 0
    assert c[0, :, :, 0].tolist() == [[0, 1], [4, 5], [4, 5], [0, 2], [8, 9], [10, 11]]
    assert wt.tolist() == [[9, 5, 7, 0, 0, 0], [1, 2, 3, 0, 0, 0]]
