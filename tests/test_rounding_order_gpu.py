"""The order of roundings of the norm and the rotation.

A 4-bit row jumps by a step where one last bit of the 16-bit row moves over the
middle of two codes, or moves its smallest or largest entry: so every operation of
the norm and the rotation is rounded by itself, in the order of the formula, and
rows and codes are those of elementary fp32 operations, bit for bit:
  sum: entries 32 apart, one after the other, then neighbours, pairs of pairs, ..;
  (x rsqrt(sum / D + eps)) w;  a c - b s, b c + a s: two products, then the sum.
"""

import pytest

from _paged import dt, make_cache

pytestmark = pytest.mark.gpu


def _sum(x):
    a = x[..., :32]
    for k in range(32, x.shape[-1], 32):
        a = a + x[..., k:k + 32]
    while a.shape[-1] > 1:
        a = a[..., 0::2] + a[..., 1::2]
    return a


def _plain(x, w, cos, sin, pos, eps, inter):
    import torch

    y = x.float()
    if eps is not None:
        y = y * torch.rsqrt(_sum(y.square()) / y.shape[-1] + eps)
        if w is not None:
            y = y * w.float()
    if cos is not None:
        c, s = (t[pos.clamp(min=0).long()][:, :, None] for t in (cos, sin))
        half = c.shape[-1]
        one = slice(0, 2 * half, 2) if inter else slice(0, half)
        two = slice(1, 2 * half, 2) if inter else slice(half, 2 * half)
        a, b = y[..., one].clone(), y[..., two].clone()
        y[..., one], y[..., two] = a * c - b * s, b * c + a * s
    return torch.where((pos >= 0)[:, :, None, None], y.to(x.dtype), torch.zeros_like(x))


def _pack(x):
    """Codes and (step, low) of 16-bit rows, by elementary fp32 operations."""
    import torch

    xf = x.float()
    low = xf.amin(-1, keepdim=True).bfloat16().float()
    step = ((xf.amax(-1, keepdim=True) - low) / torch.full_like(low, 15.0)).bfloat16().float()
    code = ((xf - low) / step).round().clamp(0, 15).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), torch.cat((step, low), -1).bfloat16()


@pytest.mark.parametrize("D,dtype,rot,inter,weights", [
    (128, "bf16", 128, False, "f32"), (64, "f16", 64, False, "f32"), (64, "f16", 32, True, "f32"),
    (128, "f16", 64, True, "own"), (128, "bf16", 16, False, None), (64, "bf16", 0, False, "own"),
    (128, "f16", 128, True, "f32"), (64, "f16", 48, False, "f32"), (128, "f16", 112, False, "f32")])
@pytest.mark.parametrize("B,M,H,G", [(2, 600, 3, 2), (1, 2600, 66, 8), (40, 1, 16, 2)])
def test_rows_and_codes(B, M, H, G, D, dtype, rot, inter, weights):
    import torch

    from nsa_block_selection_gb300 import kv_append, qk_norm_rope, rope_tables

    g = torch.Generator(device="cuda").manual_seed(B + M + D + rot)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x = (1.5 * rand(B, M, H + 2 * G, D)).to(dt(dtype))
    q, k, v = x[:, :, :H], x[:, :, H:H + G], x[:, :, H + G:]
    wq, wk = ((1 + 0.2 * rand(D)).to(torch.float32 if weights == "f32" else x.dtype) if weights else None
              for _ in range(2))
    cos, sin = rope_tables(M + 7, rot) if rot else (None, None)
    pos = torch.randperm(M + 7, generator=g, device="cuda")[:M].expand(B, M).int().contiguous()
    pos[0, M // 2:M // 2 + (M > 1)] = -1
    want = [_plain(t, w, cos, sin, pos, 1e-6, inter) for t, w in ((q, wq), (k, wk))]
    for got, y in zip(qk_norm_rope(q, k, wq, wk, cos, sin, pos, interleaved=inter), want):
        assert torch.equal(got.view(torch.int16), y.view(torch.int16))
    cols = -(-(M + 7) // 64)
    table = torch.randperm(B * cols, generator=g, device="cuda").view(B, cols).int()
    b, m = torch.nonzero(pos >= 0, as_tuple=True)
    at = pos[b, m].long()
    page, off = table[b, at // 64].long(), at % 64
    for bits in (16, 4):
        cache = make_cache(g, B * cols, 64, G, D, dtype, 16, fill=0.0)
        if bits == 4:
            from nsa_block_selection_gb300 import kv_cache

            cache = kv_cache(B * cols, 64, G, D, bits=4)
        for eps in (1e-6, None):
            w = (wq, wk) if eps is not None else (None, None)
            y = want if eps is not None else [_plain(t, None, cos, sin, pos, None, inter) for t in (q, k)]
            got = kv_append(q, k, v, cache, table, pos, *w, cos, sin, eps=eps, interleaved=inter)
            assert torch.equal(got.view(torch.int16), y[0].view(torch.int16))
            for name, rows in (("k", y[1][b, m]), ("v", v[b, m])):
                if bits == 16:
                    assert torch.equal(getattr(cache, name)[page, off], rows)
                    continue
                codes, scale = _pack(rows)
                assert torch.equal(getattr(cache, name)[page, off], codes)
                assert torch.equal(getattr(cache, name + "_scale")[page, :, off], scale)


def test_queries_turned_in_place_in_part():
    """A part of the head turned (the sum's entries are loaded again), Q where it lies."""
    import torch

    from nsa_block_selection_gb300 import kv_append, kv_cache, rope_tables

    g = torch.Generator(device="cuda").manual_seed(4)
    for D, B, M, H in ((64, 2, 500, 6), (128, 1, 2600, 40)):
        q, k = (torch.randn((B, M, n, D), generator=g, device="cuda").half() for n in (H, 2))
        cos, sin = rope_tables(M, 32)
        pos = torch.arange(M, device="cuda").expand(B, M).int().contiguous()
        want = _plain(q, None, cos, sin, pos, 1e-6, False)
        cols = -(-M // 64)
        table = torch.arange(B * cols, device="cuda").view(B, cols).int()
        kv_append(q, k, k, kv_cache(B * cols, 64, 2, D, dtype=torch.float16), table, pos, cos=cos, sin=sin,
                  q_out=q)
        assert torch.equal(q, want)
