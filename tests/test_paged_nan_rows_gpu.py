"""Rows of a 4-bit cache that are not finite, as new tokens."""

import pytest

from _paged import dt, make_cache
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


@pytest.mark.parametrize("D,dtype", [(64, "f16"), (128, "bf16")])
@pytest.mark.parametrize("M,H,G", [(2, 8, 2), (3, 8, 2), (8, 16, 2), (150, 2, 2)])
@pytest.mark.parametrize("what", ["k", "v"])
def test_a_four_bit_row_that_is_not_finite_reaches_only_its_queries(what, M, H, G, D, dtype):
    """A new token whose row is not finite is stored as NaN: the queries before it,
    in its row tile or not, do not see it."""
    import torch

    from nsa_block_selection_gb300 import kv_append

    g = torch.Generator(device="cuda").manual_seed(M)
    cache = make_cache(g, 12, 32, G, D, dtype, 4)
    table = torch.randperm(12, generator=g, device="cuda")[:10].view(1, 10).int()
    pos = torch.arange(300 - M, 300, device="cuda").view(1, M).int()
    q = torch.randn((1, M, H, D), generator=g, device="cuda").to(dt(dtype))
    clean = _attn(q, cache, table, pos, -1, 0)
    row = torch.randn((1, 1, G, D), generator=g, device="cuda").to(dt(dtype))
    bad = row.clone()
    bad[0, 0, 0, 5] = float("nan")
    kv_append(None, bad if what == "k" else row, bad if what == "v" else row, cache, table,
              pos[:, M // 2:M // 2 + 1].contiguous(), eps=None)
    o, lse = _attn(q, cache, table, pos, -1, 0)
    n, first = M // 2, H // G  # queries before it; heads of the KV head that it is in
    assert torch.equal(o[:, :n], clean[0][:, :n]) and torch.equal(lse[:, :, :n], clean[1][:, :, :n])
    assert torch.isnan(o[:, n:, :first]).all() and torch.isfinite(o[:, n:, first:]).all()
