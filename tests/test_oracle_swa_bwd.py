"""Pins of the sliding-window backward oracle: central differences of the
forward oracle, closed forms, and the identities of a softmax."""

import numpy as np
import pytest

import oracle.swa as W


def _problem(seed, B=1, M=5, N=6, H=4, G=2, D=3):
    rng = np.random.default_rng(seed)
    return (rng.standard_normal((B, M, H, D)), rng.standard_normal((B, N, G, D)),
            rng.standard_normal((B, N, G, D)), rng.standard_normal((B, M, H, D)))


@pytest.mark.parametrize("window", [(-1, -1), (-1, 0), (2, 0), (1, 2), (0, -1)])
def test_gradients_against_central_differences(window):
    q, k, v, do = _problem(1)
    o, lse = W.swa_fwd(q, k, v, *window, scale=0.7)
    grads = W.swa_bwd(q, k, v, o, lse, do, *window, scale=0.7)
    h = 1e-6
    for n, x in enumerate((q, k, v)):
        for at in np.ndindex(x.shape):
            ends = []
            for step in (h, -h):
                t = [q.copy(), k.copy(), v.copy()]
                t[n][at] += step
                ends.append(np.sum(W.swa_fwd(*t, *window, scale=0.7)[0] * do))
            assert abs((ends[0] - ends[1]) / (2 * h) - grads[n][at]) < 1e-7


def test_one_visible_key():
    """Window (0, 0): p = 1, so dV = dO, and nothing moves Q or K."""
    q, k, v, do = _problem(2, N=5, H=2, G=2)
    o, lse = W.swa_fwd(q, k, v, 0, 0)
    dq, dk, dv = W.swa_bwd(q, k, v, o, lse, do, 0, 0)
    np.testing.assert_allclose(dq, 0, atol=1e-14)
    np.testing.assert_allclose(dk, 0, atol=1e-14)
    np.testing.assert_allclose(dv, do, rtol=1e-14)


def test_identities_and_rows_without_keys():
    q, k, v, do = _problem(3, M=9, N=4)
    o, lse = W.swa_fwd(q, k, v, 2, 1)  # queries 6.. see no key
    assert np.isneginf(lse[:, :, 6:]).all()
    dq, dk, dv = W.swa_bwd(q, k, v, o, lse, do, 2, 1)
    assert (dq[:, 6:] == 0).all()
    # shifting every key by the same vector leaves the softmax unchanged
    np.testing.assert_allclose(dk.sum((0, 1)), 0, atol=1e-13)
    np.testing.assert_allclose(dv.sum(1)[0].sum(0), do[0, :6].sum((0, 1)), rtol=1e-12)
    mags = W.swa_bwd(q, k, v, o, lse, do, 2, 1, magnitudes=True)
    for g, m in zip((dq, dk, dv), mags):
        assert (np.abs(g) <= m[0] + 1e-12).all()
