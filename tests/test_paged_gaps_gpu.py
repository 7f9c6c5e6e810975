"""Queries of a call whose windows leave keys between them that nobody sees: those
rows may hold anything, in every kernel of paged_attn."""

import numpy as np
import pytest

from _paged import check_attn, dt, make_cache
from _parity import poisoned

pytestmark = pytest.mark.gpu


def _attn(q, cache, table, pos, left, sinks):
    import torch

    from nsa_block_selection_gb300 import _lib, paged_attn

    B, M, H, _ = q.shape
    out, lse = poisoned(q.shape, q.dtype), poisoned((B, H, M), torch.float32)
    paged_attn(q, cache, table, pos, window=(left, 0), sinks=sinks, out=out, lse=lse)
    torch.cuda.synchronize()
    assert _lib.sync_status() == 0
    return out, lse


def _places(kind, M, rng):
    if kind == "far":  # two places, in turn
        return np.array([700 + i // 2 if i % 2 else 40 + i // 2 for i in range(M)])
    if kind == "any order":
        return rng.permutation(900)[:M]
    if kind == "small gaps":  # windows of 4 keys, 6 apart
        return 3 + 6 * np.arange(M)
    return np.where(np.arange(M) == M - 1, 890, -1)  # padding but for the last


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("D,dtype", [(64, "f16"), (128, "bf16")])
@pytest.mark.parametrize("M,H,G", [(2, 8, 2), (3, 8, 2), (5, 16, 2), (17, 1, 1), (40, 6, 2), (150, 2, 2)])
@pytest.mark.parametrize("kind", ["far", "any order", "small gaps", "padding"])
@pytest.mark.parametrize("left,sinks", [(3, 0), (30, 5)])
def test_rows_between_windows_may_hold_anything(left, sinks, kind, M, H, G, D, dtype, bits):
    import torch

    rng = np.random.default_rng(M + left)
    g = torch.Generator(device="cuda").manual_seed(M)
    page, n = 32, 960
    cols = n // page
    cache = make_cache(g, 2 * cols + 1, page, G, D, dtype, bits)
    table = torch.randperm(2 * cols + 1, generator=g, device="cuda")[:2 * cols].view(2, cols).int()
    pos = np.stack([_places(kind, M, rng) for _ in range(2)]).astype(np.int32)
    pos = torch.from_numpy(pos).cuda()
    q = torch.randn((2, M, H, D), generator=g, device="cuda").to(dt(dtype))
    clean = _attn(q, cache, table, pos, left, sinks)
    check_attn(q, cache, table, pos, left, sinks, None, *clean, dtype)
    j = torch.arange(n, device="cuda")
    p = pos.long()[:, :, None]
    see = ((j <= p) & ((j >= p - left) | (j < sinks))).any(1)  # [2, n]
    seen = torch.zeros((2 * cols + 1, page), dtype=torch.bool, device="cuda")
    for b in range(2):
        seen[table[b].long()[:, None], (j % page).view(cols, page)] = see[b].view(cols, page)
    for fill, low in ((float("nan"), float("inf")), (3e38 if dtype == "bf16" else 60000.0, -3e38)):
        if bits == 16:
            cache.k[~seen], cache.v[~seen] = fill, fill if fill != fill else -float("inf")
        else:
            for s in (cache.k_scale, cache.v_scale):
                t = s.transpose(1, 2)
                t[..., 0][~seen], t[..., 1][~seen] = fill, low
        for x, y in zip(clean, _attn(q, cache, table, pos, left, sinks)):
            assert torch.equal(x, y)
