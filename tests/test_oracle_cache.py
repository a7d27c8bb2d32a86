"""Pins of the rope, cache and cache-attention oracles: closed forms and identities (CPU)."""

from __future__ import annotations

import numpy as np
import pytest

import oracle


def _tables(sections):
    freq = np.concatenate([10000.0 ** (-np.arange(n) / max(1, n)) for n in sections])
    return freq, np.repeat(np.arange(len(sections)), sections)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_by_hand_and_back(interleaved):
    freq, axis = _tables([1, 1])
    x = np.arange(1.0, 7.0).reshape(1, 1, 1, 6)  # R = 4, two channels copied
    pos = np.array([0.5, -1.25]).reshape(2, 1, 1)
    y = oracle.rope(x, pos, freq, axis, interleaved)
    a, b = ((0, 1), (2, 3)) if interleaved else ((0, 2), (1, 3))
    for (i, j), p in ((a, 0.5), (b, -1.25)):
        assert y[0, 0, 0, i] == pytest.approx(x[0, 0, 0, i] * np.cos(p) - x[0, 0, 0, j] * np.sin(p), abs=1e-15)
        assert y[0, 0, 0, j] == pytest.approx(x[0, 0, 0, j] * np.cos(p) + x[0, 0, 0, i] * np.sin(p), abs=1e-15)
    assert np.array_equal(y[..., 4:], x[..., 4:])
    np.testing.assert_allclose(oracle.rope(y, pos, freq, axis, interleaved, inverse=True), x, atol=1e-14)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_inverse_is_the_gradient(interleaved):
    """dL/dX of L = <Y, G> by central differences equals the inverse turn of G."""
    rng = np.random.default_rng(1)
    freq, axis = _tables([2, 1, 1])
    x, g = rng.standard_normal((2, 1, 2, 1, 10))
    pos = rng.integers(0, 1000, (3, 1, 2)).astype(np.float64)
    grad = oracle.rope(g[None, 0], pos, freq, axis, interleaved, inverse=True)
    for at in np.ndindex(*x[None, 0].shape):
        d = np.zeros_like(x[None, 0])
        d[at] = 1e-3  # L is linear in X: the difference is exact but for rounding
        up, down = (oracle.rope(x[None, 0] + s * d, pos, freq, axis, interleaved) for s in (1, -1))
        assert ((up - down) * g[None, 0]).sum() / 2e-3 == pytest.approx(grad[at], abs=1e-9)


def test_rope_depends_on_relative_positions():
    rng = np.random.default_rng(2)
    freq, axis = _tables([16, 24, 24])
    q, k = rng.standard_normal((2, 1, 1, 1, 128))
    p, r = rng.integers(0, 500, (2, 3, 1, 1)).astype(np.float64)

    def dot(shift):
        a, b = oracle.rope(q, p + shift, freq, axis), oracle.rope(k, r + shift, freq, axis)
        return float((a * b).sum())

    assert dot(0.0) == pytest.approx(dot(17.0), abs=1e-10)


def test_cells_hold_vectors_to_half_a_step():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((5, 3, 128))
    x[2, 1] = 0.0
    codes, scale = oracle.cache_write(x)
    assert np.all(scale[2, 1] == 0) and np.all(codes[2, 1] == 0)
    back = oracle.cache_value(codes, scale)
    # each rotated channel is off by half a step at most, and the rotation keeps the norm
    off = np.linalg.norm(back - x, axis=-1)
    assert np.all(off <= 0.5 * scale.astype(np.float64) * np.sqrt(128) * (1 + 1e-6) + 1e-12)


def test_seen_keys():
    assert oracle.seen(5, 2).tolist() == [[True, True, True, True, False], [True] * 5]
    tree = np.array([0b001, 0b011, 0b101])  # two branches under the first draft
    assert oracle.seen(4, 3, tree)[2].tolist() == [True, True, False, True]
    assert oracle.seen(0, 1).shape == (1, 0)
    assert not oracle.seen(2, 3, np.zeros(3, int)).any()
    # more new tokens than keys: the first ones are not in the cache
    assert oracle.seen(1, 3).tolist() == [[False], [False], [True]]


def test_cache_attention_matches_the_dense_oracle():
    """With every key seen and the values' quantisation undone, the dense INT8 attention."""
    rng = np.random.default_rng(4)
    q, k, v = rng.standard_normal((3, 6, 2, 128))
    kc, ks = oracle.cache_write(k.transpose(1, 0, 2))
    vc, vs = oracle.cache_write(v.transpose(1, 0, 2))
    o, w, _, _ = oracle.cache_attention(q, kc, ks, vc, vs, np.ones((6, 6), bool), 0.1)
    held = oracle.cache_value(vc, vs)
    for h in range(2):
        np.testing.assert_allclose(o[:, h], oracle.attention_int8(q[:, h], k[:, h], held[h], 0.1), atol=1e-12)
    np.testing.assert_allclose(w.sum(-1), 1.0, atol=1e-12)


def test_cache_attention_without_keys_is_zero():
    o, w, _, _ = oracle.cache_attention(np.ones((1, 2, 128)), np.zeros((1, 0, 128), np.int8), np.zeros((1, 0)),
                                        np.zeros((1, 0, 128), np.int8), np.zeros((1, 0)), oracle.seen(0, 1), 0.1)
    assert not o.any() and w.shape == (1, 2, 0)
