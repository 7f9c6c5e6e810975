"""nsa_swa_bwd with fp16 inputs over their whole range.

dS = p (dP - delta) is rounded to fp16 for its products whatever its size, so it
is carried times a power of two, taken from the data. A row of dQ and a row of
dK each have their own: with
    bound_i = |dO_i| max|v_j| + |delta_i|,       j over the key tiles of the row,
    bound_j = |v_j| max|dO_i| + max|delta_i|,    i over the query blocks of the key,
(Euclidean norms) which |dP - delta| never passes, the largest 2^e <= 2^40 with
bound 2^e < 2^15. Entries under fp16's 2^-14 then have the step 2^-24: half of
it, 2^-25 2^-e <= 2^-39 bound (2^-65 at least), is what a term may be off
by beside its relative half step 2^-11. The other terms of the bounds are those
of test_swa_bwd_gpu.py's head.

Expected values: the float64 oracle on the same O and LSE.
"""

import numpy as np
import pytest

import oracle.swa as W
from test_swa_bwd_gpu import _np, _problem, _run

pytestmark = pytest.mark.gpu

U = 2.0 ** -11


def _flush(n, window, scale):
    """What dQ and dK may be off by through small dS: per row or key the half
    step above, times the sum of |k| (|q|) over what it sees."""
    q, k, v, o, lse, do = n
    B, M, H, D = q.shape
    N, G = k.shape[1:3]
    nq, nv = np.sqrt((do ** 2).sum(-1)), np.sqrt((v ** 2).sum(-1))
    delta = np.abs((do * o).sum(-1))
    live = ~np.isneginf(lse).transpose(0, 2, 1)
    nq, delta = nq * live, np.where(live, delta, 0.0)
    see = np.zeros((M, N), bool)
    for i in range(M):
        see[i, W.window_keys(i, N, *window)] = True
    fq, fk = np.zeros(q.shape), np.zeros(k.shape)
    for b in range(B):
        for g in range(G):
            heads = slice(g * (H // G), (g + 1) * (H // G))
            for i0 in range(0, M, 128):  # every 128-key tile that the 128 queries touch
                rows = slice(i0, min(i0 + 128, M))
                tiles = sorted({j // 128 for j in np.flatnonzero(see[rows].any(0))})
                top = max((nv[b, 128 * t:128 * t + 128, g].max() for t in tiles), default=0.0)
                step = np.maximum((nq[b, rows, heads] * top + delta[b, rows, heads]) * 2.0 ** -39, 2.0 ** -65)
                fq[b, rows, heads] = step[..., None] * (see[rows].astype(float) @ np.abs(k[b, :, g]))[:, None]
            for j0 in range(0, N, 128):  # every 64-query block that the 128 keys touch
                keys = slice(j0, min(j0 + 128, N))
                touched = np.flatnonzero(see[:, keys].any(1))
                if touched.size == 0:
                    continue
                rows = slice(touched[0] // 64 * 64, touched[-1] // 64 * 64 + 64)
                step = nv[b, keys, g] * nq[b, rows, heads].max() + delta[b, rows, heads].max()
                step = np.maximum(step * 2.0 ** -39, 2.0 ** -65)
                qs = np.abs(q[b, :, heads]).sum(1)
                fk[b, keys, g] = step[:, None] * (see[:, keys].T.astype(float) @ qs)
    return scale * fq, scale * fk


def _check(t, window, out, grad, what=""):
    n = [_np(x) for x in t]
    D = n[0].shape[-1]
    want = W.swa_bwd(*n, *window)
    mags = W.swa_bwd(*n, *window, magnitudes=True)
    ug = 0.0 if grad == "f32" else U
    hpg = n[0].shape[2] // n[1].shape[2]
    smag = max((D ** -0.5 * np.abs(n[0][:, :, h]) @ np.abs(n[1][:, :, h // hpg]).transpose(0, 2, 1)).max()
               for h in range(n[0].shape[2]))
    ep = 2.0 ** -16 * smag + 2.0 ** -20
    store = 0.0 if grad == "f32" else 2.0 ** -25
    for name, got, w, m, f in zip(("dQ", "dK"), out, want, mags, _flush(n, window, D ** -0.5)):
        got = _np(got)
        assert np.isfinite(got).all(), f"{what} {name}: non-finite"
        err, bound = np.abs(got - w), U * m[0] + ug * np.abs(w) + (ep + 2.0 ** -15) * m[1] + f + store
        assert (err <= bound).all(), f"{what} {name}: {(err / np.maximum(bound, 1e-300)).max():.2f} x bound"
    got, bound = _np(out[2]), U * mags[2][0] + ug * np.abs(want[2]) + (ep + U * ug) * mags[2][0] + store
    # (p 2^12 has fp16's step 2^-24 below 2^-14: half of it, 2^-37, for each row)
    bound = bound + 2.0 ** -37 * np.abs(n[5]).sum((1, 2))[:, None, None]
    assert (np.abs(got - want[2]) <= bound).all(), f"{what} dV"


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [(7, 0), (-1, -1)])
@pytest.mark.parametrize("do_scale", [2.0 ** -20, 2.0 ** -12, 1.0, 50.0, 200.0, 2.0 ** 12])
def test_scales_of_the_incoming_gradient(D, window, do_scale):
    t = _problem(2, 300, 300, 4, 2, D, "f16", window, 41, do_scale=do_scale)
    _check(t, window, _run(t, window, "f16", "f32"), "f32")
    if do_scale == 200.0:  # gradients that fp16 holds
        _check(t, window, _run(t, window, "f16"), None)


def _scaled(scales_v, scales_do, window, seed, M=640, H=2, D=64):
    """V's and dO's rows times factors of their own, with the forward of that V."""
    import torch

    from nsa_block_selection_gb300 import swa_fwd

    q, k, v, _, _, do = _problem(1, M, M, H, 1, D, "f16", window, seed)
    col = lambda s: torch.as_tensor(s, device="cuda").view(1, M, 1, 1)  # noqa: E731
    v, do = (v.float() * col(scales_v)).half(), (do.float() * col(scales_do)).half()
    o, lse = swa_fwd(q, k, v, window=window)
    assert torch.isfinite(o).all()
    return q, k, v, o, lse, do


@pytest.mark.parametrize("D", [64, 128])
def test_large_rows_beside_small_ones(D):
    """dO of a few rows 2^26 times that of the others, and V of a few keys 2^10
    times: rows and keys whose tiles hold none of them keep all their bits."""
    M = 640
    for which in ("do", "v", "both"):
        sv, sd = np.ones(M, np.float32), np.full(M, 2.0 ** -14, np.float32)
        if which != "v":
            sd[300:303] = 2.0 ** 12
        if which != "do":
            sv[[10, 400]] = 2.0 ** 10
        t = _scaled(sv, sd, (40, 0), 42, D=D)
        _check(t, (40, 0), _run(t, (40, 0), "f16", "f32"), "f32", which)


def test_cut_tiles():
    """Parts of a tile choose their powers of two each for itself."""
    for M, N, window in ((130, 2500, (0, -1)), (2500, 130, (-1, -1)), (1300, 1300, (-1, 0))):
        t = _problem(1, M, N, 2, 1, 64, "f16", window, 43, do_scale=300.0)
        _check(t, window, _run(t, window, "f16", "f32"), "f32", f"{M}x{N}")


def test_rows_without_keys_and_hidden_rows_do_not_count():
    """What dO holds in rows without keys, and V in keys that no query sees,
    infinities and NaN among it, changes nothing."""
    import torch

    from nsa_block_selection_gb300 import swa_bwd

    window = (5, 5)
    t = _problem(1, 330, 300, 2, 1, 64, "f16", window, 44, do_scale=2.0 ** -12)
    want = swa_bwd(*t, window=window, grad_dtype=torch.float32)
    do = t[5].clone()
    do[:, 306:] = 60000.0  # (finite, as rows that share a tile with live ones must be)
    for a, b in zip(want, swa_bwd(*t[:5], do, window=window, grad_dtype=torch.float32)):
        assert torch.equal(a, b)
    t = _problem(1, 100, 128, 2, 1, 64, "f16", window, 45, do_scale=2.0 ** -12)
    want = swa_bwd(*t, window=window, grad_dtype=torch.float32)
    for bad in (float("nan"), float("inf")):
        v = t[2].clone()
        v[:, 110:] = bad
        got = swa_bwd(*t[:2], v, *t[3:], window=window, grad_dtype=torch.float32)
        for a, b in zip(want, got):
            assert torch.equal(a, b)


def test_no_gradient_is_none():
    import torch

    from nsa_block_selection_gb300 import swa_bwd

    t = _problem(1, 200, 200, 2, 1, 128, "f16", (30, 0), 46)
    for x in swa_bwd(*t[:5], torch.zeros_like(t[5]), window=(30, 0)):
        assert (x == 0).all()


def test_captured_calls_follow_new_gradients():
    """A replay takes its powers of two from what the tensors hold then."""
    import torch

    from nsa_block_selection_gb300 import _lib, swa_bwd

    window = (100, 0)
    t = _problem(1, 400, 400, 4, 2, 128, "f16", window, 47, do_scale=2.0 ** -12)
    out = [torch.empty_like(x, dtype=torch.float32) for x in t[:3]]
    ws = torch.empty(_lib.swa_bwd_workspace_bytes(1, 400, 400, 4, 2, 128, window),
                     dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        swa_bwd(*t, window=window, dq=out[0], dk=out[1], dv=out[2], workspace=ws)
    for seed, do_scale in ((48, 2.0 ** 11), (49, 2.0 ** -12)):
        u = _problem(1, 400, 400, 4, 2, 128, "f16", window, seed, do_scale=do_scale)
        for a, b in zip(t, u):
            a.copy_(b)
        for x in out:
            x.fill_(float("nan"))
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, _run(u, window, "f16", "f32")):
            assert torch.equal(a, b)
        _check(u, window, out, "f32")
