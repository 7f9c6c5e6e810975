"""The norm and rotation of long prompts with many heads, against the float64
oracle with the bounds of test_norm_rope_gpu.py.

A token whose heads take more than 8 groups of row slots (32 heads at D = 128,
64 at D = 64) and a call of more than 128 x 152 = 19,456 groups go to a kernel
of their own, in which a warp walks a token's heads, or a segment of them
where the tokens are fewer than 16 x 152 = 2432.
"""

import pytest

from test_norm_rope_gpu import _case, _check_fwd

pytestmark = pytest.mark.gpu

WALKED = [
    # B, M, H, G, D, dtype, rot, interleaved, pad, weights
    # 17 groups a token; 2 segments of 36 rows, the second from Q's last rows into K
    (2, 610, 61, 5, 128, "bf16", 128, False, True, "f32"),
    # 18 groups; 36 rows are two rounds of 16 in flight and a quarter of one
    (1, 1500, 64, 8, 128, "f16", 64, True, True, "f16"),
    # segments of 24 and 17, Q's last 13 rows and K's 4 in the second
    (3, 650, 37, 4, 128, "bf16", 0, False, True, None),
    # whole tokens: 9 and 10 groups
    (2, 1300, 64, 8, 64, "f16", 64, True, True, "f32"),
    (1, 2600, 66, 7, 64, "bf16", 32, False, False, "bf16"),
]


def _walked(B, M, H, G, D):
    slots = 32 // (D // 16)
    groups = -(-(H + G) // slots)
    return groups > 8 and B * M * groups > 128 * 152


@pytest.mark.parametrize("B,M,H,G,D,dtype,rot,inter,pad,weights", WALKED)
def test_walked_heads(B, M, H, G, D, dtype, rot, inter, pad, weights):
    """Views of a projection in, rows with room around them out, then in place."""
    import torch

    from nsa_block_selection_gb300 import qk_norm_rope

    assert _walked(B, M, H, G, D)
    case = _case(B, M, H, G, D, dtype, rot, 61, fused=True, pad=pad, weights=weights)
    q, k, wq, wk, cos, sin, pos = case
    if pad:  # padding is not read
        dead = (pos < 0) | (pos >= (cos.shape[0] if rot else 2 ** 31 - 1))
        q[dead], k[dead] = float("nan"), float("inf")
        assert dead.any()
    wide = torch.full((B, M + 1, H + G + 3, D), 7.0, device="cuda", dtype=q.dtype)
    outs = wide[:, :M, 1:1 + H], wide[:, :M, 2 + H:2 + H + G]
    qk_norm_rope(q, k, wq, wk, cos, sin, pos, eps=1e-5, interleaved=inter, q_out=outs[0],
                 k_out=outs[1])
    if pad:  # (the oracle gives zeros there)
        clean = tuple(torch.where(dead[..., None, None], torch.zeros_like(x), x) for x in (q, k))
    else:
        clean = q, k
    _check_fwd(clean + case[2:], dtype, 1e-5, inter, *outs)
    assert (wide[:, M] == 7).all() and (wide[:, :, [0, H + 1, H + G + 2]] == 7).all()
    qk_norm_rope(q, k, wq, wk, cos, sin, pos, eps=1e-5, interleaved=inter, q_out=q, k_out=k)
    assert torch.equal(q, outs[0]) and torch.equal(k, outs[1])


@pytest.mark.parametrize("H,G,D,M", [(64, 8, 128, 1200), (64, 8, 64, 2200)])
def test_both_sides_of_the_threshold(H, G, D, M):
    """The same tokens in a call that walks heads and in calls that do not: both
    within a rounding of the oracle, so within two of one another."""
    import torch

    from nsa_block_selection_gb300 import qk_norm_rope, rope_tables

    g = torch.Generator(device="cuda").manual_seed(62)
    q, k = (1.5 * torch.randn(1, M, n, D, generator=g, device="cuda").bfloat16() for n in (H, G))
    wq, wk = (1 + 0.3 * torch.randn(D, generator=g, device="cuda") for _ in range(2))
    cos, sin = rope_tables(M, D)
    pos = torch.randperm(M, generator=g, device="cuda").int()
    assert _walked(1, M, H, G, D) and not _walked(1, M // 2, H, G, D)
    whole = qk_norm_rope(q, k, wq, wk, cos, sin, pos)
    for i in (0, M // 2):
        half = slice(i, i + M // 2)
        part = qk_norm_rope(q[:, half], k[:, half], wq, wk, cos, sin, pos[half].contiguous())
        for a, b in zip(whole, part):
            a, b = a[:, half].float(), b.float()
            # half a step each, and 2 x 24 x 2^-24 of two terms, together under 20
            assert ((a - b).abs() <= 2 * 2.0 ** -8 * b.abs() + 2.0 ** -14).all()


def test_a_captured_walk_follows_its_inputs():
    import torch

    from nsa_block_selection_gb300 import qk_norm_rope

    case = _case(1, 1200, 64, 8, 128, "bf16", 128, 63)
    q, k, wq, wk, cos, sin, pos = case
    out = torch.empty_like(q), torch.empty_like(k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    qk_norm_rope(q, k, wq, wk, cos, sin, pos, q_out=out[0], k_out=out[1], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    _check_fwd(case, "bf16", 1e-6, False, *out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qk_norm_rope(q, k, wq, wk, cos, sin, pos, q_out=out[0], k_out=out[1])
    q.copy_(torch.randn(q.shape, device="cuda"))  # 3 segments of 24 rows a token
    pos.copy_(pos.flip(1))
    for x in out:
        x.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    _check_fwd(case, "bf16", 1e-6, False, *out)
