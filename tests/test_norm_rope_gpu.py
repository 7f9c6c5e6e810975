"""nsa_qk_norm_rope and nsa_qk_norm_rope_bwd against the float64 oracle.

Tolerances, per element, from the unit roundoffs u = eps/2 of the stored type
and e = 2^-24 of the fp32 arithmetic, with the oracle's magnitudes |.| (every
term made positive):

* forward: u |y| for the store (half of the smallest subnormal for tiny
  values) and 24 e |terms|: the sum of squares is a chain of 16 fused steps
  and 3 exchanges (19 e, halved by the root), the root at most 2 steps of its
  type (4 e), 1/D, eps and three products (5 e), the turn's two products and
  sum (2 e);
* dx: u |dx| and 60 e |terms|: g (2 e), g w (1 e), its row sum (19 e), r three
  times (3 x 15 e at most, halved where it meets the sum), the last products;
* dw: a chain of n terms is off by at most (n + 30) e sum|terms|, n the
  longest chain of one lane and the joins after it.
"""

import numpy as np
import pytest

import oracle.norm_rope as R
from _parity import poisoned

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25}  # half of the smallest subnormal


def _dt(name):
    import torch

    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[name]


def _np(t):
    return t.detach().double().cpu().numpy()


def _close(got, want, mag, u, tiny, steps, what):
    err, bound = np.abs(got - want), u * np.abs(want) + tiny + steps * E * mag
    assert np.isfinite(got).all(), f"{what}: non-finite"
    assert (err <= bound).all(), f"{what}: {(err / np.maximum(bound, 1e-300)).max():.2f} x bound"


def _case(B, M, H, G, D, dtype, rot, seed, fused=False, pad=False, weights="f32", rows=None):
    import torch

    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _dt(dtype)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    if fused:
        x = (1.5 * rand(B, M, H + 2 * G, D)).to(dt)
        q, k = x[:, :, :H], x[:, :, H:H + G]
    else:
        q, k = (1.5 * rand(B, M, H, D)).to(dt), (1.5 * rand(B, M, G, D)).to(dt)
    wq = wk = None
    if weights:
        wq, wk = ((1 + 0.3 * rand(D)).to(_dt(weights)) for _ in range(2))
    rows = rows or M + 5
    cos = sin = None
    if rot:
        from nsa_block_selection_gb300 import rope_tables

        cos, sin = rope_tables(rows, rot)
    pos = torch.randint(0, rows, (B, M), generator=g, device="cuda", dtype=torch.int32)
    if pad:
        for b in range(B):
            pos[b, M - (b + 1) * M // 3:] = -1 if b % 2 == 0 else rows + b
    return q, k, wq, wk, cos, sin, pos


def _oracle_args(w, cos, sin, pos):
    return (None if w is None else _np(w), None if cos is None else _np(cos),
            None if sin is None else _np(sin), None if pos is None else pos.cpu().numpy())


def _check_fwd(case, dtype, eps, inter, q_out, k_out):
    q, k, wq, wk, cos, sin, pos = case
    for what, x, w, y in (("q", q, wq, q_out), ("k", k, wk, k_out)):
        w_, c_, s_, p_ = _oracle_args(w, cos, sin, pos)
        want = R.norm_rope(_np(x), w_, c_, s_, p_, eps, inter)
        mag = R.norm_rope(_np(x), w_, c_, s_, p_, eps, inter, magnitudes=True)
        _close(_np(y), want, mag, U[dtype], TINY[dtype], 24, what)


def _chain(B, M, heads, D):
    """The longest chain of additions: a lane's rows (8 heads' worth of warps at
    least share the tokens), 3 exchanges, 8 warps, 456 / 32 partials, 5 exchanges."""
    rows = 32 // (D // 16)
    return -(-B * M // 8) * -(-heads // rows) + 3 + 8 + 15 + 5


def _check_bwd(case, grads, dtype, eps, inter, out):
    q, k, wq, wk, cos, sin, pos = case
    for what, x, w, dy, dx, dw in (("q", q, wq, grads[0], out[0], out[2]),
                                   ("k", k, wk, grads[1], out[1], out[3])):
        w_, c_, s_, p_ = _oracle_args(w, cos, sin, pos)
        args = (_np(x), w_, _np(dy), c_, s_, p_, eps, inter)
        want, want_w = R.norm_rope_bwd(*args)
        mag, mag_w = R.norm_rope_bwd(*args, magnitudes=True)
        _close(_np(dx), want, mag, U[dtype], TINY[dtype], 60, "d" + what)
        if dw is not None:
            n = _chain(x.shape[0], x.shape[1], x.shape[2], x.shape[3])
            _close(_np(dw), want_w, mag_w, 0.0, 0.0, n + 30, "dw" + what)


SHAPES = [
    # B, M, H, G, D, dtype, rot, interleaved, fused, pad, weights
    (1, 1, 64, 8, 128, "bf16", 128, False, True, False, "f32"),
    (5, 1, 8, 1, 64, "f16", 64, True, False, False, "f16"),
    (2, 130, 3, 1, 128, "bf16", 64, False, True, True, "bf16"),
    (3, 77, 7, 5, 64, "f16", 32, True, True, True, "f32"),
    (1, 700, 16, 2, 128, "f16", 16, False, False, False, None),
    (1, 257, 1, 1, 64, "bf16", 48, False, False, False, "f32"),
    (2, 33, 6, 2, 128, "bf16", 0, False, True, True, "f32"),
    (1, 5000, 8, 2, 64, "bf16", 64, False, True, False, "f32"),
]


@pytest.mark.parametrize("B,M,H,G,D,dtype,rot,inter,fused,pad,weights", SHAPES)
def test_forward_matches_oracle(B, M, H, G, D, dtype, rot, inter, fused, pad, weights):
    from nsa_block_selection_gb300 import qk_norm_rope

    case = _case(B, M, H, G, D, dtype, rot, 3, fused, pad, weights)
    q, k, wq, wk, cos, sin, pos = case
    out = qk_norm_rope(q, k, wq, wk, cos, sin, pos, eps=1e-5, interleaved=inter,
                       q_out=poisoned(q.shape, q.dtype), k_out=poisoned(k.shape, k.dtype))
    _check_fwd(case, dtype, 1e-5, inter, *out)


@pytest.mark.parametrize("grad", ["same", "f32"])
@pytest.mark.parametrize("B,M,H,G,D,dtype,rot,inter,fused,pad,weights", SHAPES)
def test_backward_matches_oracle(B, M, H, G, D, dtype, rot, inter, fused, pad, weights, grad):
    import torch

    from nsa_block_selection_gb300 import qk_norm_rope_bwd

    case = _case(B, M, H, G, D, dtype, rot, 4, fused, pad, weights)
    q, k, wq, wk, cos, sin, pos = case
    gt = q.dtype if grad == "same" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(5)
    grads = [(0.1 * torch.randn(x.shape, generator=g, device="cuda")).to(gt) for x in (q, k)]
    out = qk_norm_rope_bwd(q, k, *grads, wq, wk, cos, sin, pos, eps=1e-5, interleaved=inter,
                           dq=poisoned(q.shape, q.dtype), dk=poisoned(k.shape, k.dtype),
                           dq_weight=poisoned((D,), torch.float32),
                           dk_weight=poisoned((D,), torch.float32))
    _check_bwd(case, grads, dtype, 1e-5, inter, out)
    again = qk_norm_rope_bwd(q, k, *grads, wq, wk, cos, sin, pos, eps=1e-5, interleaved=inter)
    for a, b in zip(out, again):  # a fixed order of every sum
        assert torch.equal(a, b)


FEW = [
    # heads of a token that fill, share, or run over the row slots of a warp
    (1, 1, 64), (2, 1, 64), (3, 2, 64), (4, 4, 64), (5, 3, 64), (20, 12, 64),
    (1, 1, 128), (2, 2, 128), (3, 1, 128), (9, 2, 128),
]


@pytest.mark.parametrize("H,G,D", FEW)
@pytest.mark.parametrize("B,M,dtype,rot,inter", [(1, 1, "bf16", 64, False), (3, 5, "f16", 32, True),
                                                 (2, 601, "bf16", 64, False)])
def test_few_heads(B, M, dtype, rot, inter, H, G, D):
    """Several tokens to a warp: partial groups, padding among them, outputs
    with room around every row, which stays as it was."""
    import torch

    from nsa_block_selection_gb300 import qk_norm_rope, qk_norm_rope_bwd

    case = _case(B, M, H, G, D, dtype, rot, 21, pad=M > 1)
    q, k, wq, wk, cos, sin, pos = case
    room = [torch.full((B, M + 1, h + 1, D), 7.0, device="cuda", dtype=q.dtype)
            for h in (H, G, H, G)]
    outs = [t[:, :M, :h] for t, h in zip(room, (H, G, H, G))]
    qk_norm_rope(q, k, wq, wk, cos, sin, pos, eps=1e-5, interleaved=inter, q_out=outs[0],
                 k_out=outs[1])
    _check_fwd(case, dtype, 1e-5, inter, outs[0], outs[1])
    g = torch.Generator(device="cuda").manual_seed(22)
    for grad in (dtype, "f32"):
        grads = [torch.randn(x.shape, generator=g, device="cuda").to(_dt(grad)) for x in (q, k)]
        out = qk_norm_rope_bwd(q, k, *grads, wq, wk, cos, sin, pos, eps=1e-5,
                               interleaved=inter, dq=outs[2], dk=outs[3])
        _check_bwd(case, grads, dtype, 1e-5, inter, out)
    for t, h in zip(room, (H, G, H, G)):
        assert (t[:, M:] == 7).all() and (t[:, :, h:] == 7).all()


def test_positions_by_default_shared_and_far():
    import torch

    from nsa_block_selection_gb300 import qk_norm_rope

    case = _case(2, 50, 4, 2, 128, "bf16", 128, 6, rows=70000)
    q, k, wq, wk, cos, sin, _ = case
    run = lambda pos: qk_norm_rope(q, k, wq, wk, cos, sin, pos)  # noqa: E731
    ar = torch.arange(50, device="cuda", dtype=torch.int32)
    for a, b in zip(run(None), run(ar)):
        assert torch.equal(a, b)
    for a, b in zip(run(ar), run(ar.expand(2, 50).contiguous())):
        assert torch.equal(a, b)
    far = ar + 69950
    _check_fwd(case[:6] + (far.expand(2, 50),), "bf16", 1e-6, False, *run(far))


def test_in_place_and_strided_outputs():
    """Outputs over the inputs, and written into slices whose neighbours stay."""
    import torch

    from nsa_block_selection_gb300 import qk_norm_rope, qk_norm_rope_bwd

    q, k, wq, wk, cos, sin, pos = _case(2, 61, 6, 2, 128, "bf16", 64, 7, fused=True, pad=True)
    want = qk_norm_rope(q, k, wq, wk, cos, sin, pos)
    wide = torch.full((2, 61, 12, 128), 7.0, dtype=q.dtype, device="cuda")
    qk_norm_rope(q, k, wq, wk, cos, sin, pos, q_out=wide[:, :, 1:7], k_out=wide[:, :, 8:10])
    assert torch.equal(wide[:, :, 1:7], want[0]) and torch.equal(wide[:, :, 8:10], want[1])
    assert (wide[:, :, [0, 7, 10, 11]] == 7).all()
    fused = torch.cat((q, k), 2)
    a, b = fused[:, :, :6], fused[:, :, 6:]
    grads = torch.randn(a.shape, device="cuda").to(q.dtype), torch.randn(b.shape, device="cuda").to(q.dtype)
    ref = qk_norm_rope_bwd(q, k, *grads, wq, wk, cos, sin, pos)
    over = qk_norm_rope_bwd(q, k, *grads, wq, wk, cos, sin, pos, dq=grads[0], dk=grads[1])
    for x, y in zip(ref, over):
        assert torch.equal(x, y)
    qk_norm_rope(a, b, wq, wk, cos, sin, pos, q_out=a, k_out=b)
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])


def test_padding_is_never_read_and_special_rows():
    """NaN in padding tokens and their gradients stays out of everything; a
    row of zeros, a row with an infinity and a huge row keep to themselves."""
    import torch

    from nsa_block_selection_gb300 import qk_norm_rope, qk_norm_rope_bwd

    q, k, wq, wk, cos, sin, pos = _case(2, 40, 4, 2, 64, "bf16", 64, 8, pad=True)
    dead = (pos < 0) | (pos >= cos.shape[0])
    assert dead.any() and not dead.all()
    q[dead] = float("nan")
    k[dead] = float("inf")
    g = [torch.randn(x.shape, device="cuda").to(q.dtype) for x in (q, k)]
    for t in g:
        t[dead] = float("nan")
    y = qk_norm_rope(q, k, wq, wk, cos, sin, pos)
    d = qk_norm_rope_bwd(q, k, *g, wq, wk, cos, sin, pos)
    for t in (*y, *d):
        assert torch.isfinite(t).all()
    for t in (*y, *d[:2]):
        assert (t[dead] == 0).all()
    clean = y[0].clone()
    q[0, 0, 1] = 0.0
    q[0, 1, 2, 5] = float("inf")
    q[0, 2, 3] = 1e30  # its squares pass the largest fp32
    y = qk_norm_rope(q, k, wq, wk, cos, sin, pos)[0]
    assert (y[0, 0, 1] == 0).all()
    assert torch.isnan(y[0, 1, 2]).any()
    touched = torch.zeros(y.shape[:3], dtype=torch.bool, device="cuda")
    touched[0, 0, 1] = touched[0, 1, 2] = touched[0, 2, 3] = True
    assert torch.equal(y[~touched], clean[~touched])


def test_without_weight_gradients_and_empty():
    import torch

    from nsa_block_selection_gb300 import qk_norm_rope, qk_norm_rope_bwd

    q, k, wq, wk, cos, sin, pos = _case(1, 30, 4, 2, 64, "f16", 64, 9)
    g = [torch.randn(x.shape, device="cuda").half() for x in (q, k)]
    a = qk_norm_rope_bwd(q, k, *g, wq, wk, cos, sin, pos)
    b = qk_norm_rope_bwd(q, k, *g, wq, wk, cos, sin, pos, weight_grads=False)
    assert b[2] is None and b[3] is None
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    e = q[:, :0], k[:, :0]
    out = qk_norm_rope(*e, wq, wk, cos, sin)
    assert out[0].shape == e[0].shape
    out = qk_norm_rope_bwd(*e, *e, wq, wk, cos, sin, dq_weight=poisoned((64,), torch.float32))
    assert (out[2] == 0).all() and (out[3] == 0).all()


def test_refusals_on_the_device():
    import torch

    from nsa_block_selection_gb300 import NsaError, qk_norm_rope

    q, k, wq, wk, cos, sin, pos = _case(1, 30, 4, 2, 64, "f16", 64, 10)
    with pytest.raises(NsaError):  # fewer table rows than tokens
        qk_norm_rope(q, k, wq, wk, cos[:29].contiguous(), sin[:29].contiguous())
    with pytest.raises(NsaError):  # 40 rotated entries
        qk_norm_rope(q, k, wq, wk, cos[:, :20].contiguous(), sin[:, :20].contiguous(), pos)
    with pytest.raises(NsaError):  # rows that start at odd multiples of 2 bytes
        x = torch.zeros(1, 30, 4, 65, device="cuda").half()[..., :64]
        qk_norm_rope(x, k, wq, wk, cos, sin, pos)
    for bad in (dict(positions=pos.long()), dict(q_weight=wq.double()), dict(cos=cos.half())):
        with pytest.raises(TypeError):
            qk_norm_rope(**dict(dict(q=q, k=k, q_weight=wq, k_weight=wk, cos=cos, sin=sin,
                                     positions=pos), **bad))
    for bad in (dict(sin=None), dict(positions=pos[:, :29]), dict(q_weight=wq[:32]),
                dict(q_out=torch.empty(1, 30, 4, 64).half()), dict(k=k.transpose(2, 3))):
        with pytest.raises(ValueError):
            qk_norm_rope(**dict(dict(q=q, k=k, q_weight=wq, k_weight=wk, cos=cos, sin=sin,
                                     positions=pos), **bad))


def test_another_stream_and_graph_replay():
    """The calls run on the stream they are given, and a captured pair of
    calls replays on new contents of the same tensors."""
    import torch

    from nsa_block_selection_gb300 import _lib, qk_norm_rope, qk_norm_rope_bwd

    q, k, wq, wk, cos, sin, pos = _case(2, 90, 4, 2, 128, "bf16", 128, 11)
    g = [torch.randn(x.shape, device="cuda").to(q.dtype) for x in (q, k)]
    yo = torch.empty_like(q), torch.empty_like(k)
    do = [torch.empty_like(q), torch.empty_like(k)] + [torch.empty(128, device="cuda") for _ in range(2)]
    ws = torch.empty(_lib.norm_rope_bwd_workspace_bytes(2, 90, 128), dtype=torch.uint8, device="cuda")

    def both(stream=None):
        qk_norm_rope(q, k, wq, wk, cos, sin, pos, q_out=yo[0], k_out=yo[1], stream=stream)
        qk_norm_rope_bwd(q, k, *g, wq, wk, cos, sin, pos, dq=do[0], dk=do[1], dq_weight=do[2],
                         dk_weight=do[3], workspace=ws, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    both(side)
    torch.cuda.current_stream().wait_stream(side)
    _check_fwd((q, k, wq, wk, cos, sin, pos), "bf16", 1e-6, False, *yo)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    q.copy_(torch.randn(q.shape, device="cuda"))
    for t in (*yo, *do):
        t.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    case = (q, k, wq, wk, cos, sin, pos)
    _check_fwd(case, "bf16", 1e-6, False, *yo)
    _check_bwd(case, g, "bf16", 1e-6, False, do)


def test_batched_prefix_past_32_bit_offsets():
    """A projection whose rows start past 2^31 elements: the last batch of a
    strided view, against the same rows on their own."""
    import torch

    from nsa_block_selection_gb300 import qk_norm_rope

    B, M, H, G, D = 2, 4, 4, 2, 128
    big = torch.empty(2 ** 31 + 2 ** 20, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((B, M, H + G, D), (2 ** 31, (H + G) * D, D, 1))
    x.copy_(torch.randn(B, M, H + G, D, device="cuda"))
    cos, sin = __import__("nsa_block_selection_gb300").rope_tables(M, D)
    a = qk_norm_rope(x[:, :, :H], x[:, :, H:], None, None, cos, sin)
    y = x.contiguous()
    b = qk_norm_rope(y[:, :, :H], y[:, :, H:], None, None, cos, sin)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
