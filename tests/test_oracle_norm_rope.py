"""Pins of the norm-and-rotation oracle: closed forms, invariants, and its
gradients against central differences (everything in float64)."""

import numpy as np
import pytest

import oracle.norm_rope as R


def _tables(rows, rot, base=100.0):
    half = rot // 2
    ang = np.arange(rows)[:, None] * base ** (-np.arange(half) / max(half, 1))
    return np.cos(ang), np.sin(ang)


def test_hand_worked_row():
    x = np.array([3.0, 0.0, 4.0, 0.0]).reshape(1, 1, 1, 4)  # mean of squares 25/4
    cos, sin = np.array([[1.0, 1.0], [0.0, 1.0]]), np.array([[0.0, 0.0], [1.0, 0.0]])
    w = np.array([1.0, 2.0, 10.0, 4.0])
    y = R.norm_rope(x, w, cos, sin, [[1]], 0.0, False)  # pair (0, 2) a quarter turn
    np.testing.assert_allclose(y[0, 0, 0], [-16.0, 0.0, 1.2, 0.0], atol=1e-14)
    y = R.norm_rope(x, w, cos, sin, [[1]], 0.0, True)   # pair (0, 1) a quarter turn
    np.testing.assert_allclose(y[0, 0, 0], [0.0, 1.2, 16.0, 0.0], atol=1e-14)


@pytest.mark.parametrize("interleaved", [False, True])
def test_a_turn_is_orthogonal_and_depends_on_position_differences(interleaved):
    rng = np.random.default_rng(0)
    cos, sin = _tables(40, 16)
    q, k = rng.standard_normal((2, 1, 1, 1, 16))
    dots = []
    for a, b in ((7, 3), (30, 26), (4, 0)):
        x = R.norm_rope(q, None, cos, sin, [[a]], 0.0, interleaved)
        y = R.norm_rope(k, None, cos, sin, [[b]], 0.0, interleaved)
        np.testing.assert_allclose(np.sum(x * x), 16.0, rtol=1e-13)
        dots.append(np.sum(x * y))
    np.testing.assert_allclose(dots, dots[0], rtol=1e-12)


def test_partial_rotation_position_zero_and_padding():
    rng = np.random.default_rng(1)
    cos, sin = _tables(10, 8)
    x = rng.standard_normal((2, 3, 2, 16))
    pos = [[0, 4, -1], [10, 9, 0]]  # -1 and 10 are outside the table
    y = R.norm_rope(x, None, cos, sin, pos, 1e-6, False)
    n = R.norm_rope(x, None, None, None, None, 1e-6, False)
    np.testing.assert_array_equal(y[0, 2], 0.0)
    np.testing.assert_array_equal(y[1, 0], 0.0)
    np.testing.assert_allclose(y[0, 0], n[0, 0], rtol=1e-15)
    np.testing.assert_allclose(y[0, 1, :, 8:], n[0, 1, :, 8:], rtol=1e-15)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 4, 8])
def test_gradients_against_central_differences(interleaved, rot):
    rng = np.random.default_rng(2)
    x, dy = rng.standard_normal((2, 2, 3, 2, 8))
    w = rng.standard_normal(8) + 1
    cos, sin = _tables(5, rot) if rot else (None, None)
    pos = [[0, -1, 3], [4, 2, 2]]
    args = (cos, sin, pos, 1e-2, interleaved)
    dx, dw = R.norm_rope_bwd(x, w, dy, *args)

    def loss(x_, w_):
        return np.sum(R.norm_rope(x_, w_, *args) * dy)

    h = 1e-6
    for at in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[at] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[at]) < 1e-7
    for j in range(8):
        e = np.zeros(8)
        e[j] = h
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[j]) < 1e-7
    # dx is orthogonal to x up to the part that eps takes
    dx0, _ = R.norm_rope_bwd(x, w, dy, cos, sin, pos, 0.0, interleaved)
    np.testing.assert_allclose(np.sum(dx0 * x, -1), 0.0, atol=1e-12)
    mx, mw = R.norm_rope_bwd(x, w, dy, *args, magnitudes=True)
    assert (mx >= np.abs(dx) - 1e-12).all() and (mw >= np.abs(dw) - 1e-12).all()
