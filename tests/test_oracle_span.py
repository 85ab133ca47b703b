"""The span and rope oracle against the dense oracle, closed forms and invariants (CPU)."""

import math

import numpy as np

import oracle
from oracle import span as ref


def test_all_keys_is_dense_attention():
    rng = np.random.default_rng(0)
    q, k, v = (rng.standard_normal((2, n, 3, 64)) for n in (9, 9, 9))
    o, lse, w = ref.span_attention(q, k, v)
    do, dl = oracle.dense_attention(q, k, v)
    np.testing.assert_allclose(o, do, atol=1e-12)
    np.testing.assert_allclose(lse, dl, atol=1e-12)
    assert (w >= np.abs(o) - 1e-12).all()


def test_prefix_equals_concatenated_keys_and_grouped_heads_share():
    rng = np.random.default_rng(1)
    q = rng.standard_normal((2, 4, 4, 64))
    k, v = rng.standard_normal((2, 2, 5, 2, 64))
    kp, vp = rng.standard_normal((2, 3, 2, 64))
    a = ref.span_attention(q, k, v, k_prefix=kp, v_prefix=vp, slopes=np.full(4, 0.1), cap=3.0)
    both = [np.concatenate([np.broadcast_to(p, (2, 3, 2, 64)), x], 1) for p, x in ((kp, k), (vp, v))]
    b = ref.span_attention(q, *(np.repeat(x, 2, 2) for x in both), slopes=np.full(4, 0.1), cap=3.0)
    np.testing.assert_allclose(a[0], b[0], atol=1e-12)
    np.testing.assert_allclose(a[1], b[1], atol=1e-12)


def test_empty_and_single_key_rows():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((3, 1, 2, 1, 64))
    o, lse, _ = ref.span_attention(q, k, v, spans=np.array([[1, 1], [1, 2]]))
    assert (o[0, 0] == 0).all() and lse[0, 0, 0] == -np.inf
    np.testing.assert_allclose(o[0, 1], v[0, 1])
    np.testing.assert_allclose(lse[0, 0, 1], q[0, 1, 0] @ k[0, 1, 0] / 8.0)


def test_rope_keeps_lengths_and_relative_products():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((1, 2, 1, 64))
    freq, axis = [10.0 ** (-i / 8) for i in range(32)], [i % 2 for i in range(32)]
    at = lambda p: np.array(p, dtype=float).reshape(1, 2, 2)
    for pairing in ("interleaved", "half"):
        a = ref.rope(x, at([[3, 5], [7, 8]]), freq, axis, pairing)
        b = ref.rope(x, at([[103, 105], [-13, -12]]), freq, axis, pairing)
        np.testing.assert_allclose(np.linalg.norm(a, axis=-1), np.linalg.norm(x, axis=-1))
        np.testing.assert_allclose(a[0, 0, 0] @ a[0, 1, 0], b[0, 0, 0] @ b[0, 1, 0], atol=1e-9)
    y = ref.rope(x, at([[0, 0], [0, 0]]), freq, axis, "half", weight=np.full(64, 2.0), eps=0.0)
    np.testing.assert_allclose(np.sqrt((y ** 2).mean(-1)), 2.0)


def test_grid_positions():
    assert ref.grid_positions((3, 2, 4), 7, 3).tolist() == [[0, 1, 1], [1, 0, 0], [3, 0, 1]]
    assert math.prod((3, 2, 4)) == 24
