"""nsa_swa_bwd against the float64 oracle, which takes the same O and LSE.

Per element, with u the unit roundoff of the inputs' type (fp16 2^-11, bf16
2^-8), the stored type's u_g (0 for fp32) and the oracle's positive sums:

* dV: u sum p |dO| (p rounded before its product), u_g |dV|, and the error of
  p itself: relative to p, the fp32 score (128 products added with at most a
  step of 2^-23 each: 2^-16 scale |q|.|k|) plus 2^-20 for LSE in base 2, the
  fused multiply and the exponential;
* dQ, dK: u sum |dS| |k| (|q|), u_g |dQ|, and, relative to p (|dO|.|v| +
  |dO|.|O|), the error of p, of dP (2^-16) and of delta (2^-17).

Sums over m terms in fp32 add 2^-23 m of the same magnitudes at most: 2^-13
covers 1000 terms; they are far below it in these problems.
"""

import numpy as np
import pytest

import oracle.swa as W
from _parity import poisoned

pytestmark = pytest.mark.gpu

U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def _dt(name):
    import torch

    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[name]


def _np(t):
    return t.detach().double().cpu().numpy()


def _problem(B, M, N, H, G, D, dtype, window, seed, scale=None, do_scale=1.0):
    import torch

    from nsa_block_selection_gb300 import swa_fwd

    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(_dt(dtype))  # noqa: E731
    q, k, v = rand(B, M, H, D), rand(B, N, G, D), rand(B, N, G, D)
    do = (do_scale * torch.randn((B, M, H, D), generator=g, device="cuda")).to(_dt(dtype))
    o, lse = swa_fwd(q, k, v, window=window, scale=scale)
    return q, k, v, o, lse, do


def _run(t, window, dtype, grad=None, **kw):
    import torch

    from nsa_block_selection_gb300 import _lib, swa_bwd

    q, k, v, o, lse, do = t
    gt = _dt(grad or dtype)
    out = swa_bwd(q, k, v, o, lse, do, window=window, dq=poisoned(q.shape, gt),
                  dk=poisoned(k.shape, gt), dv=poisoned(k.shape, gt), **kw)
    torch.cuda.synchronize()
    assert _lib.sync_status() == 0
    return out


def _check(t, window, dtype, out, grad=None, scale=None, what="", flush=0.0):
    """flush: the smallest step of the type, where results may fall below it."""
    n = [_np(x) for x in t]
    want = W.swa_bwd(*n, *window, scale=scale)
    mags = W.swa_bwd(*n, *window, scale=scale, magnitudes=True)
    u, ug = U[dtype], 0.0 if grad == "f32" else U[dtype]
    sc = scale or n[0].shape[-1] ** -0.5
    qk = sc * np.abs(n[0]).sum(-1).max() * np.abs(n[1]).max() if n[1].size else 0.0
    hpg = n[0].shape[2] // n[1].shape[2]
    smag = 0.0
    for h in range(n[0].shape[2]):
        smag = max(smag, sc * (np.abs(n[0][:, :, h]) @ np.abs(n[1][:, :, h // hpg]).transpose(0, 2, 1)).max())
    assert smag <= qk + 1e-9
    ep = 2.0 ** -16 * smag + 2.0 ** -20
    for name, got, w, m in zip(("dQ", "dK", "dV"), out, want, mags):
        got = _np(got)
        assert np.isfinite(got).all(), f"{what} {name}: non-finite"
        bound = u * m[0] + ug * np.abs(w) + flush
        bound += (ep + u * ug) * m[0] if name == "dV" else (ep + 2.0 ** -15) * m[1]
        err = np.abs(got - w)
        assert (err <= bound).all(), \
            f"{what} {name}: {(err / np.maximum(bound, 1e-300)).max():.2f} x bound"


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("window", [(-1, -1), (-1, 0), (100, 0), (0, 0), (37, 53), (300, -1)])
def test_every_element(D, dtype, window):
    t = _problem(2, 520, 520, 4, 2, D, dtype, window, 20 + D)
    _check(t, window, dtype, _run(t, window, dtype), what=f"{window}")


@pytest.mark.parametrize("M,N", [(1, 1), (1, 700), (63, 64), (64, 63), (65, 129), (128, 128),
                                 (129, 257), (300, 520), (520, 300), (130, 1000), (1000, 127)])
@pytest.mark.parametrize("window", [(64, 0), (-1, 0), (10, 200), (-1, -1)])
def test_lengths(M, N, window):
    t = _problem(1, M, N, 4, 1, 128, "bf16", window, 7)
    _check(t, window, "bf16", _run(t, window, "bf16"), what=f"{M}x{N} {window}")


CUT = [
    # few query tiles and many keys, and the other way: both kernels cut into
    # parts, some without a step (a causal window's short tiles)
    (1, 1, 4100, 1, 1, 64, "bf16", (-1, -1)),
    (1, 130, 2500, 3, 1, 128, "f16", (0, -1)),
    (2, 200, 3000, 2, 2, 128, "bf16", (-1, 2000)),
    (1, 2100, 2100, 1, 1, 128, "bf16", (-1, 0)),
    (1, 2050, 2049, 2, 1, 64, "f16", (5, -1)),
    (1, 4100, 40, 8, 1, 128, "bf16", (-1, -1)),
    (1, 1500, 5, 3, 1, 64, "bf16", (100, 1400)),
]


@pytest.mark.parametrize("B,M,N,H,G,D,dtype,window", CUT)
@pytest.mark.parametrize("grad", ["f32", None])
def test_cut_tiles(B, M, N, H, G, D, dtype, window, grad):
    import torch

    t = _problem(B, M, N, H, G, D, dtype, window, 31)
    out = _run(t, window, dtype, grad)
    _check(t, window, dtype, out, grad, what=f"{M}x{N} {window}")
    for x, y in zip(out, _run(t, window, dtype, grad)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("H,G", [(4, 4), (6, 2), (3, 1), (16, 1), (5, 5)])
@pytest.mark.parametrize("grad", ["f32", None])
def test_head_groups_scale_and_fp32_gradients(H, G, grad):
    t = _problem(1, 260, 260, H, G, 64, "bf16", (90, 10), 8, scale=0.2)
    out = _run(t, (90, 10), "bf16", grad, scale=0.2)
    _check(t, (90, 10), "bf16", out, grad, scale=0.2)


@pytest.mark.parametrize("D", [64, 128])
def test_fp32_gradients_round_to_the_16_bit_ones(D):
    import torch

    t = _problem(1, 400, 400, 8, 2, D, "f16", (128, 0), 9)
    a, b = _run(t, (128, 0), "f16", "f32"), _run(t, (128, 0), "f16")
    for x, y in zip(a, b):
        assert torch.equal(x.half(), y)


def test_small_gradients_keep_their_precision_in_fp16():
    """A thousand visible keys and a small dO: p and dS lie where fp16 has
    few bits left; the carried powers of two keep them exact to 2^-11. What
    remains is the smallest step of fp16 where a gradient itself falls
    below 2^-14 (stored as fp32 here: none)."""
    t = _problem(1, 1100, 1100, 2, 1, 128, "f16", (-1, -1), 10, do_scale=2.0 ** -7)
    _check(t, (-1, -1), "f16", _run(t, (-1, -1), "f16", "f32"), "f32",
           # dS' = 2^6 dS has the step 2^-24: half of it per term, 1100 terms
           # of |k|, |q| <= 5, times scale, 2^-6
           flush=0.5 * 2.0 ** -24 * 2.0 ** -6 * 1100 * 5 * 128 ** -0.5)


def test_rows_without_keys_and_keys_without_queries():
    import torch

    t = _problem(1, 700, 300, 4, 2, 64, "bf16", (5, 5), 11)  # queries 306.. see nothing
    assert torch.isneginf(t[4][:, :, 306:]).all()
    out = _run(t, (5, 5), "bf16")
    assert (out[0][:, 306:] == 0).all()
    _check(t, (5, 5), "bf16", out)
    t = _problem(1, 100, 600, 4, 2, 128, "bf16", (5, 5), 12)  # keys 105.. are not seen
    out = _run(t, (5, 5), "bf16")
    assert (out[1][:, 105:] == 0).all() and (out[2][:, 105:] == 0).all()
    _check(t, (5, 5), "bf16", out)


def test_empty_problems():
    import torch

    from nsa_block_selection_gb300 import swa_bwd

    q = torch.randn(1, 200, 4, 64, device="cuda").bfloat16()
    k = torch.zeros(1, 0, 2, 64, device="cuda").bfloat16()
    lse = torch.full((1, 4, 200), float("-inf"), device="cuda")
    dq, dk, dv = swa_bwd(q, k, k, q, lse, q, dq=poisoned(q.shape, q.dtype))
    assert (dq == 0).all() and dk.numel() == 0
    e = q[:, :0]
    k = torch.randn(1, 50, 2, 64, device="cuda").bfloat16()
    dq, dk, dv = swa_bwd(e, k, k, e, lse[:, :, :0], e, dk=poisoned(k.shape, torch.float32),
                         dv=poisoned(k.shape, torch.float32), grad_dtype=torch.float32)
    assert (dk == 0).all() and (dv == 0).all() and dq.numel() == 0


@pytest.mark.parametrize("D", [64, 128])
def test_hidden_pairs_may_hold_anything_within_range(D):
    """Hidden scores that overflow to infinity and V rows of NaN past every
    query's window leave the gradients of the others unchanged."""
    import torch

    from nsa_block_selection_gb300 import swa_bwd

    q, k, v, o, lse, do = _problem(1, 256, 256, 2, 1, D, "bf16", (40, 0), 13)
    want = swa_bwd(q[:, :200].contiguous(), k[:, :200].contiguous(), v[:, :200].contiguous(),
                   o[:, :200].contiguous(), lse[:, :, :200].contiguous(), do[:, :200].contiguous(),
                   window=(40, 0))
    q, k, v, o, lse, do = (x[:, :200].contiguous() if x.dim() == 4 else x[:, :, :200].contiguous()
                           for x in (q, k, v, o, lse, do))
    k2 = torch.cat((k, torch.full_like(k[:, :56], 3e37)), 1)
    v2 = torch.cat((v, torch.full_like(v[:, :56], float("nan"))), 1)
    got = swa_bwd(q, k2, v2, o, lse, do, window=(40, 0))
    assert torch.equal(got[0], want[0])
    assert torch.equal(got[1][:, :200], want[1]) and torch.equal(got[2][:, :200], want[2])
    assert (got[1][:, 200:] == 0).all() and (got[2][:, 200:] == 0).all()


def test_equal_calls_give_equal_bits_on_any_stream_and_in_a_graph():
    import torch

    from nsa_block_selection_gb300 import _lib, swa_bwd

    window = (256, 0)
    t = _problem(1, 1000, 1000, 8, 2, 128, "bf16", window, 14)
    want = _run(t, window, "bf16")
    for a, b in zip(want, _run(t, window, "bf16")):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = swa_bwd(*t, window=window, stream=side)
    main = swa_bwd(*t, window=window)  # at the same time, workspaces of their own
    torch.cuda.synchronize()
    for a, b, c in zip(want, got, main):
        assert torch.equal(a, b) and torch.equal(a, c)
    ws = torch.empty(_lib.swa_bwd_workspace_bytes(1, 1000, 1000, 8, 2, 128, window),
                     dtype=torch.uint8, device="cuda")
    out = [torch.empty_like(x) for x in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        swa_bwd(*t, window=window, dq=out[0], dk=out[1], dv=out[2], workspace=ws)
    u = _problem(1, 1000, 1000, 8, 2, 128, "bf16", window, 15)
    want = _run(u, window, "bf16")
    for a, b in zip(t, u):
        a.copy_(b)
    for x in out:
        x.fill_(float("nan"))
    ws.fill_(255)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, out):
        assert torch.equal(a, b)


@pytest.mark.parametrize("D,window", [(128, (512, 0)), (128, (-1, 0)), (64, (1000, 300))])
def test_large_sampled(D, window):
    """M = N = 4096, H = 16, H_kv = 2: one KV head's rows of sampled queries
    and keys from the definition (fp64 on the GPU)."""
    import torch

    M, H, G = 4096, 16, 2
    t = _problem(1, M, M, H, G, D, "bf16", window, 16)
    out = _run(t, window, "bf16")
    q, k, v, o, lse, do = (x.double() for x in t)
    i, j = torch.arange(M, device="cuda")[:, None], torch.arange(M, device="cuda")[None]
    see = torch.ones(M, M, dtype=torch.bool, device="cuda")
    if window[0] >= 0:
        see &= j >= i - window[0]
    if window[1] >= 0:
        see &= j <= i + window[1]
    dk, dv, mk, mv, fk = (torch.zeros(M, D, dtype=torch.float64, device="cuda") for _ in range(5))
    g, sc, u, smag = 1, D ** -0.5, U["bf16"], 0.0
    kh, vh = k[0, :, g], v[0, :, g]
    for h in range(8, 16):
        smag = max(smag, float(sc * (q[0, :, h].abs() @ kh.abs().T).max()))
    # the bounds of the file's head. fp32 errors are relative to `wide`, not
    # to dS: query 0 of a causal window has one key, dP - delta cancels to an
    # exact 0 there, and an error of dP or delta (2^-16, 2^-17) is all that is left
    ep = 2.0 ** -16 * smag + 2.0 ** -20
    for h in range(8, 16):
        qh, oh, dh = q[0, :, h], o[0, :, h], do[0, :, h]
        p = torch.where(see, torch.exp(sc * (qh @ kh.T) - lse[0, h][:, None]), 0.0)
        ds = p * (dh @ vh.T - (dh * oh).sum(-1, keepdim=True))
        wide = p * (dh.abs() @ vh.abs().T + (dh * oh).abs().sum(-1, keepdim=True))
        dq = sc * ds @ kh
        bound = u * (sc * ds.abs() @ kh.abs() + dq.abs()) + (ep + 2.0 ** -15) * sc * wide @ kh.abs()
        assert ((out[0][0, :, h].double() - dq).abs() <= bound).all(), h
        dk += sc * ds.T @ qh
        mk += sc * ds.abs().T @ qh.abs()
        fk += sc * wide.T @ qh.abs()
        dv += p.T @ dh
        mv += p.T @ dh.abs()
    bound = u * (mk + dk.abs()) + (ep + 2.0 ** -15) * fk
    assert ((out[1][0, :, g].double() - dk).abs() <= bound).all()
    bound = u * (mv + dv.abs()) + (ep + u * u) * mv
    assert ((out[2][0, :, g].double() - dv).abs() <= bound).all()


def test_offsets_past_32_bits():
    """More than 2^31 entries of Q: the last queries against the same rows on
    their own (a slice that starts at a multiple of both tiles, so that every
    sum is the same one)."""
    import torch

    from nsa_block_selection_gb300 import swa_bwd

    M, H, D, window, cut = 131_200, 128, 128, (64, 0), 130_560
    g = torch.Generator(device="cuda").manual_seed(18)
    big = [torch.empty(1, M, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    q, o, do = (t.normal_(generator=g) for t in big)
    k, v = (torch.randn(1, M, 1, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    lse = torch.full((1, H, M), 8.0, device="cuda")
    assert q.numel() > 2 ** 31
    a = swa_bwd(q, k, v, o, lse, do, window=window)
    tail = [t[:, cut:].contiguous() for t in (q, k, v, o)] + [lse[:, :, cut:].contiguous(),
                                                             do[:, cut:].contiguous()]
    b = swa_bwd(*tail, window=window)
    assert torch.equal(a[0][:, cut + 128:], b[0][:, 128:])  # (whose windows lie in the slice)
    assert torch.isfinite(a[0][:, cut + 128:]).all() and a[0][:, -1].abs().max() > 0
    for x, y in ((a[1], b[1]), (a[2], b[2])):
        # the last tiles may be cut into other parts: one rounding apart
        x, y = x[:, cut:].float(), y.float()
        assert ((x - y).abs() <= 2.0 ** -7 * y.abs().clamp(min=1e-3)).all()


def test_own_stream_allocations():
    """On a side stream, what the call allocates and drops is not handed to the
    current stream's work while the side stream still runs."""
    import torch

    from nsa_block_selection_gb300 import swa_bwd

    t = _problem(1, 2000, 2000, 8, 2, 128, "bf16", (300, 0), 19)
    want = swa_bwd(*t, window=(300, 0))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    busy = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            for _ in range(4):
                busy = busy @ busy  # the side stream is late
        got = swa_bwd(*t, window=(300, 0), stream=side)
        junk = [torch.full((1 << 22,), float("nan"), device="cuda") for _ in range(8)]
        torch.cuda.current_stream().wait_stream(side)
        for a, b in zip(want, got):
            assert torch.equal(a, b)
        del junk


def test_refusals_on_the_device():
    import torch

    from nsa_block_selection_gb300 import NsaError, swa_bwd

    t = _problem(1, 300, 300, 4, 2, 64, "bf16", (64, 0), 17)
    with pytest.raises(NsaError):  # too small a workspace
        swa_bwd(*t, window=(64, 0), workspace=torch.empty(100, dtype=torch.uint8, device="cuda"))
    wide = torch.randn(1, 300, 8, 64, device="cuda").bfloat16()
    with pytest.raises(ValueError):  # a strided view, as in the forward
        swa_bwd(wide[:, :, :4], *t[1:], window=(64, 0))
    with pytest.raises(ValueError):
        swa_bwd(*t[:4], t[4].cpu(), t[5], window=(64, 0))
    with pytest.raises(TypeError):
        swa_bwd(*t[:5], t[5].float(), window=(64, 0))
