"""CPU oracle for the per-head RMS norm with the position rotation, and its
gradients -- TEST INFRASTRUCTURE ONLY.

Only the tests may use this module. The product path never imports or calls
it, and shares no code with it.

Per row x (one head of one token, D entries), weight w, eps, and the angles
(c_i, s_i) that the tables hold for the token's position:

* r = 1 / sqrt(mean(x^2) + eps), n = x r w;
* pair i of the first R entries -- (i, i + R/2), or (2i, 2i + 1) when
  interleaved -- goes from (a, b) to (a c_i - b s_i, b c_i + a s_i);
* a token whose position is outside the table is padding: zero rows, zero
  gradients, no share in the weight's gradient.

Plain definition in float64. The gradients follow from the chain rule: g is
dy turned back, dw = sum over rows of g x r, and with u = g w,
dx_j = r u_j - r^3 x_j sum(u x) / D.

``magnitudes=True`` returns the same sums with every term made positive: the
scale that rounding errors are measured against.
"""

from __future__ import annotations

import numpy as np

__all__ = ["turn", "norm_rope", "norm_rope_bwd"]


def turn(x: np.ndarray, c: np.ndarray, s: np.ndarray, interleaved: bool) -> np.ndarray:
    """Turn the pairs of x [..., D] by the angles (c, s) [..., R/2]."""
    half = c.shape[-1]
    y = np.array(x, dtype=np.float64)
    for i in range(half):
        p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        y[..., p] = x[..., p] * c[..., i] - x[..., q] * s[..., i]
        y[..., q] = x[..., q] * c[..., i] + x[..., p] * s[..., i]
    return y


def _angles(cos, sin, positions, B, M, R):
    pos = np.broadcast_to(np.arange(M) if positions is None else np.asarray(positions), (B, M))
    live = pos >= 0
    if R == 0:
        none = np.zeros((B, M, 1, 0))
        return none, none, live
    live = live & (pos < cos.shape[0])
    at = np.where(live, pos, 0)
    return (np.asarray(cos, np.float64)[at][:, :, None], np.asarray(sin, np.float64)[at][:, :, None],
            live)


def norm_rope(x, w, cos, sin, positions, eps, interleaved, magnitudes=False):
    """x [B, M, heads, D] -> float64 of the same shape."""
    x = np.asarray(x, np.float64)
    B, M, _, D = x.shape
    c, s, live = _angles(cos, sin, positions, B, M, 0 if cos is None else 2 * cos.shape[1])
    x = np.where(live[:, :, None, None], x, 0.0)
    w = np.ones(D) if w is None else np.asarray(w, np.float64)
    with np.errstate(divide="ignore", invalid="ignore"):
        n = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * w
    if magnitudes:
        y = turn(np.abs(n), np.abs(c), -np.abs(s), interleaved)  # |a||c| + |b||s| of the first entry
        z = turn(np.abs(n), np.abs(c), np.abs(s), interleaved)   # and of the second
        y = np.maximum(y, z)
    else:
        y = turn(n, c, s, interleaved)
    return np.where(live[:, :, None, None], y, 0.0)


def norm_rope_bwd(x, w, dy, cos, sin, positions, eps, interleaved, magnitudes=False):
    """(dx [B, M, heads, D], dw [D]), float64."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    B, M, _, D = x.shape
    c, s, live = _angles(cos, sin, positions, B, M, 0 if cos is None else 2 * cos.shape[1])
    keep = live[:, :, None, None]
    x, dy = np.where(keep, x, 0.0), np.where(keep, dy, 0.0)
    w = np.ones(D) if w is None else np.asarray(w, np.float64)
    with np.errstate(divide="ignore", invalid="ignore"):
        r = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    r = np.where(keep, r, 0.0)  # a padding token's zeros would divide by 0
    if magnitudes:
        a, ca, sa = np.abs(dy), np.abs(c), np.abs(s)
        g = np.maximum(turn(a, ca, sa, interleaved), turn(a, ca, -sa, interleaved))
        x, w = np.abs(x), np.abs(w)
        dx = r * g * w + r ** 3 * x * np.mean(g * w * x, axis=-1, keepdims=True)
    else:
        g = turn(dy, c, -s, interleaved)
        dx = r * g * w - r ** 3 * x * np.mean(g * w * x, axis=-1, keepdims=True)
    return np.where(keep, dx, 0.0), np.sum(g * (x * r), axis=(0, 1, 2))
