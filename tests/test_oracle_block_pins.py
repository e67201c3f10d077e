"""Pins of the oracle's rotary, layer norm and dropout: hand-derived values,
invariants and finite differences (CPU, 64 bits)."""
import math

import numpy as np
import pytest

from oracle import (angles, dropout, element_keep_mask, frequencies, keep_threshold, layer_norm,
                    layer_norm_backward, philox4x32_10, rotate)


def _turns(w):
    return [int(round(x / (2 * math.pi) * 2.0 ** 64)) for x in w]


def test_rotary_quarter_turn_by_hand():
    # a quarter of a turn per position: (1, 0) -> (0, 1) -> (-1, 0) -> (0, -1)
    x = np.zeros((1, 1, 4, 2))
    x[..., 0] = 1.0
    y = rotate(x, [1 << 62], np.arange(4)[None])
    assert np.allclose(y[0, 0], [[1, 0], [0, 1], [-1, 0], [0, -1]], atol=1e-15)


def test_rotary_angles_follow_the_frequencies():
    w, m = frequencies(64)
    assert m == 1.0 and w[0] == 1.0 and math.isclose(w[-1], 10000.0 ** (-62 / 64))
    p = np.array([[0, 1, 17, 4095, -3]])
    got = angles(_turns(w), p)
    want = p[..., None] * w
    assert np.abs(np.exp(1j * got) - np.exp(1j * want)).max() < 1e-11


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_invariants(interleaved):
    rng = np.random.default_rng(1)
    w, _ = frequencies(12, base=100.0)
    t = _turns(w)
    x, y = rng.standard_normal((2, 2, 3, 5, 16))
    p = rng.integers(0, 1 << 40, (2, 5))
    rx = rotate(x, t, p, 1.3, interleaved)
    # <R x, y> = <x, R^T y>, R^T R = m^2 on the rotated columns, the rest copied
    ry = rotate(y, t, p, 1.3, interleaved, adjoint=True)
    assert math.isclose((rx * y).sum(), (x * ry).sum(), rel_tol=1e-12)
    back = rotate(rx, t, p, 1.3, interleaved, adjoint=True)
    assert np.allclose(back[..., :12], 1.69 * x[..., :12], rtol=0, atol=1e-12)
    assert np.array_equal(back[..., 12:], x[..., 12:])
    # scores depend on the distance of the positions alone
    s1 = (rotate(x, t, p, 1.0, interleaved) * rotate(y, t, p + 5, 1.0, interleaved)).sum(-1)
    s2 = (rotate(x, t, p + 77, 1.0, interleaved) * rotate(y, t, p + 82, 1.0, interleaved)).sum(-1)
    assert np.allclose(s1, s2, atol=1e-12)


def test_scalings_by_hand():
    plain, _ = frequencies(8, base=256.0)
    assert np.allclose(plain, [1, 0.25, 0.0625, 0.015625])
    linear, m = frequencies(8, base=256.0, scaling="linear", factor=4.0)
    assert np.allclose(linear, plain / 4) and m == 1.0
    base, _ = frequencies(8, base=256.0, scaling="base", factor=4.0)
    assert base[0] == 1.0 and math.isclose(base[-1], plain[-1] / 4)
    # over 64 pi positions the plain frequencies make 32, 8, 2 and 0.5 turns
    ramp, m = frequencies(8, base=256.0, scaling="ramp", factor=2.0,
                          original_length=64 * math.pi, low_turns=1.0, high_turns=15.0)
    assert np.allclose(ramp, [1, 0.25 * 0.75, 0.0625 * (1 / 14 + 13 / 28), 0.015625 / 2])
    assert math.isclose(m, 1 + 0.1 * math.log(2))


def test_element_mask_is_the_generator_word_by_word():
    seed, p = 0x123456789ABCDEF0, 0.3
    got = element_keep_mask(23, seed, p)
    for e in range(23):
        w = philox4x32_10(e // 4, 0, 0, 1, seed & 0xFFFFFFFF, seed >> 32)[e % 4]
        assert got[e] == (int(w) >= keep_threshold(p))
    # beyond 2^34 elements the second counter word steps
    far = element_keep_mask(4, seed, p, first=1 << 34)
    assert [bool(v) for v in far] == [int(w) >= keep_threshold(p) for w in
                                      philox4x32_10(0, 1, 0, 1, seed & 0xFFFFFFFF, seed >> 32)]


def test_dropout_scales_and_drops():
    x = np.ones(1 << 16)
    y = dropout(x, 0.25, 7)
    assert set(np.round(np.unique(y), 12)) == {0.0, round(1 / 0.75, 12)}
    assert abs(y.mean() - 1.0) < 5 * math.sqrt(0.25 / 0.75 / x.size)
    x[:] = np.inf
    assert np.all((dropout(x, 0.25, 7) == 0) | (dropout(x, 0.25, 7) == np.inf))


def test_layer_norm_by_hand():
    y, mean, rstd = layer_norm(np.array([[1.0, 3.0], [5.0, 5.0]]), np.array([2.0, 1.0]),
                               np.array([0.0, 1.0]), 0.0 + 1e-300)
    assert np.allclose(mean, [2, 5]) and math.isclose(rstd[0], 1.0)
    assert np.allclose(y, [[-2, 2], [0, 1]])


@pytest.mark.parametrize("affine", [False, True])
def test_layer_norm_backward_against_differences(affine):
    rng = np.random.default_rng(3)
    x, dy = rng.standard_normal((2, 4, 7))
    gamma, beta = (rng.standard_normal((2, 7)) if affine else (None, None))
    eps, step = 1e-3, 1e-5

    def loss(x, gamma, beta):
        return (layer_norm(x, gamma, beta, eps)[0] * dy).sum()

    _, mean, rstd = layer_norm(x, gamma, beta, eps)
    dx, dgamma, dbeta = layer_norm_backward(dy, x, gamma, mean, rstd)
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = step
        d = (loss(x + e, gamma, beta) - loss(x - e, gamma, beta)) / (2 * step)
        assert abs(d - dx[i]) < 1e-8
    for i in range(7 if affine else 0):
        e = np.zeros(7)
        e[i] = step
        assert abs((loss(x, gamma + e, beta) - loss(x, gamma - e, beta)) / (2 * step)
                   - dgamma[i]) < 1e-8
        assert abs((loss(x, gamma, beta + e) - loss(x, gamma, beta - e)) / (2 * step)
                   - dbeta[i]) < 1e-8
