"""The operators of an attention layer run one after the other, as a training
step uses them, against fp64 autograd of the same layer:

norm and rotation -> sliding-window attention -> its gradients -> back through
the rotation and the norm (Q, K, V slices of one projection), and the same
around the selection attention with its fp32 gradients; and a step captured
into a graph.

Tolerance, on the 2-norm of each gradient relative to the exact one's: every
16-bit rounding on the way is at most u = 2^-11 relative (fp16). Q and K carry
one each into scores of at most `smag` = scale max |q|.|k| (in absolute
products), which moves p by 2 u smag; O, p, dS, dQ or dK, dV and the result
carry one each: 2 smag + 6 of them, each once.
"""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -11


def _reference(x, wq, wk, H, G, cos, sin, window, dy, eps):
    """fp64 gradients of (x, wq, wk) of the layer, by autograd."""
    import torch

    x, wq, wk = (t.detach().double().requires_grad_() for t in (x, wq, wk))
    B, M, _, D = x.shape
    half = cos.shape[1]
    c, s = cos[:M].double()[None, :, None], sin[:M].double()[None, :, None]

    def norm_turn(t, w):
        n = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + eps) * w
        a, b, rest = n[..., :half], n[..., half:2 * half], n[..., 2 * half:]
        return torch.cat((a * c - b * s, b * c + a * s, rest), -1)

    q, k, v = norm_turn(x[:, :, :H], wq), norm_turn(x[:, :, H:H + G], wk), x[:, :, H + G:]
    k, v = (t.repeat_interleave(H // G, 2) for t in (k, v))
    sc = torch.einsum("bihd,bjhd->bhij", q, k) * D ** -0.5
    smag = (torch.einsum("bihd,bjhd->bhij", q.abs(), k.abs()) * D ** -0.5).max().item()
    i, j = torch.arange(M, device="cuda")[:, None], torch.arange(M, device="cuda")[None]
    see = (j <= i) if window[0] < 0 else (j <= i) & (j >= i - window[0])
    p = torch.softmax(sc.masked_fill(~see, float("-inf")), -1)
    y = torch.einsum("bhij,bjhd->bihd", p, v)
    y.backward(dy.double())
    return y.detach(), x.grad, wq.grad, wk.grad, smag


def _close(got, want, smag, what):
    err = ((got.double() - want).norm() / want.norm()).item()
    assert err <= (2 * smag + 6) * U, f"{what}: {err:.2e} against {(2 * smag + 6) * U:.2e}"


def _layer(B, M, H, G, D, rot, seed):
    import torch

    from nsa_block_selection_gb300 import rope_tables

    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(B, M, H + 2 * G, D, generator=g, device="cuda").half()
    wq, wk = (1 + 0.2 * torch.randn(D, generator=g, device="cuda") for _ in range(2))
    dy = torch.randn(B, M, H, D, generator=g, device="cuda").half()
    return (x, wq, wk, *rope_tables(M + 3, rot), dy)


@pytest.mark.parametrize("D,rot,window", [(128, 128, (100, 0)), (64, 32, (-1, 0))])
def test_sliding_window_layer(D, rot, window):
    import torch

    from nsa_block_selection_gb300 import (qk_norm_rope, qk_norm_rope_bwd, swa_bwd, swa_fwd)

    B, M, H, G, eps = 2, 333, 8, 2, 1e-5
    x, wq, wk, cos, sin, dy = _layer(B, M, H, G, D, rot, 1)
    y, dx, dwq, dwk, smag = _reference(x, wq, wk, H, G, cos, sin, window, dy, eps)
    xq, xk, v = x[:, :, :H], x[:, :, H:H + G], x[:, :, H + G:].contiguous()
    q, k = qk_norm_rope(xq, xk, wq, wk, cos, sin, eps=eps)
    o, lse = swa_fwd(q, k, v, window=window)
    dq, dk, dv = swa_bwd(q, k, v, o, lse, dy, window=window)
    dxo = torch.full_like(x, float("nan"))  # one gradient of the projection's output
    out = qk_norm_rope_bwd(xq, xk, dq, dk, wq, wk, cos, sin, eps=eps, dq=dxo[:, :, :H],
                           dk=dxo[:, :, H:H + G])
    dxo[:, :, H + G:] = dv
    _close(o, y, smag, "y")
    for name, a, b in (("dx of q", dxo[:, :, :H], dx[:, :, :H]),
                       ("dx of k", dxo[:, :, H:H + G], dx[:, :, H:H + G]),
                       ("dx of v", dxo[:, :, H + G:], dx[:, :, H + G:]),
                       ("dwq", out[2], dwq), ("dwk", out[3], dwk)):
        _close(a, b, smag, name)


def test_selection_layer_with_fp32_gradients():
    """Every block of a row selected, so that the layer is causal attention."""
    import torch

    from nsa_block_selection_gb300 import (qk_norm_rope, qk_norm_rope_bwd, sel_attn_bwd,
                                           sel_attn_fwd)

    B, M, H, G, D, bs, eps = 1, 320, 16, 2, 128, 64, 1e-5
    x, wq, wk, cos, sin, dy = _layer(B, M, H, G, D, 128, 2)
    y, dx, dwq, dwk, smag = _reference(x, wq, wk, H, G, cos, sin, (-1, 0), dy, eps)
    xq, xk, v = x[:, :, :H], x[:, :, H:H + G], x[:, :, H + G:].contiguous()
    q, k = qk_norm_rope(xq, xk, wq, wk, cos, sin, eps=eps)
    t, c = torch.arange(M // bs, device="cuda"), torch.arange(M, device="cuda")[:, None] // bs
    idx = torch.where(t <= c, t, -1).int().view(1, M, 1, -1).expand(B, M, G, -1).contiguous()
    o, lse = sel_attn_fwd(q, k, v, idx, bs)
    dq, dk, dv = sel_attn_bwd(q, k, v, idx, o, lse, dy.float(), bs)
    out = qk_norm_rope_bwd(xq, xk, dq, dk, wq, wk, cos, sin, eps=eps)
    _close(o, y, smag, "y")
    for name, a, b in (("dx of q", out[0], dx[:, :, :H]), ("dx of k", out[1], dx[:, :, H:H + G]),
                       ("dx of v", dv, dx[:, :, H + G:]), ("dwq", out[2], dwq),
                       ("dwk", out[3], dwk)):
        _close(a, b, smag, name)


def test_a_step_in_a_graph():
    """Forward and backward of the layer captured together, replayed on new
    contents, equal to the eager step bit for bit."""
    import torch

    from nsa_block_selection_gb300 import (qk_norm_rope, qk_norm_rope_bwd, swa_bwd, swa_fwd)

    B, M, H, G, D = 1, 257, 4, 2, 64
    x, wq, wk, cos, sin, dy = _layer(B, M, H, G, D, 64, 3)

    def step():
        xq, xk, v = x[:, :, :H], x[:, :, H:H + G], x[:, :, H + G:].contiguous()
        q, k = qk_norm_rope(xq, xk, wq, wk, cos, sin)
        o, lse = swa_fwd(q, k, v, window=(64, 0))
        dq, dk, dv = swa_bwd(q, k, v, o, lse, dy, window=(64, 0))
        return (o, dv, *qk_norm_rope_bwd(xq, xk, dq, dk, wq, wk, cos, sin))

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for n in range(2):
        x.copy_(torch.randn(x.shape, device="cuda"))
        dy.copy_(torch.randn(dy.shape, device="cuda"))
        graph.replay()
        for a, b in zip(captured, step()):
            assert torch.equal(a, b), n


def test_a_decoding_step_equals_the_rows_of_a_prefill():
    """Tokens normed and turned one at a time, each at its position, give the
    bits of the whole sequence's call."""
    import torch

    from nsa_block_selection_gb300 import qk_norm_rope

    B, M, H, G, D = 3, 40, 8, 2, 128
    x, wq, wk, cos, sin, _ = _layer(B, M, H, G, D, 128, 4)
    q, k = qk_norm_rope(x[:, :, :H], x[:, :, H:H + G], wq, wk, cos, sin)
    for m in (0, 7, 39):
        pos = torch.full((B, 1), m, dtype=torch.int32, device="cuda")
        a, b = qk_norm_rope(x[:, m:m + 1, :H], x[:, m:m + 1, H:H + G], wq, wk, cos, sin, pos)
        assert torch.equal(a[:, 0], q[:, m]) and torch.equal(b[:, 0], k[:, m])
