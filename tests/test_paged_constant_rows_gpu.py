"""Rows of V that 4 bits hold without a step (zeros, constants) among others of any
size, by every kernel of paged_attn: to the bounds of _paged.py, which know no step
but the rows' own."""

import pytest

from _paged import check_attn, dt, make_cache
from _parity import poisoned

pytestmark = pytest.mark.gpu


def _attn(q, cache, table, pos):
    import torch

    from nsa_block_selection_gb300 import _lib, paged_attn

    B, M, H, _ = q.shape
    out, lse = poisoned(q.shape, q.dtype), poisoned((B, H, M), torch.float32)
    paged_attn(q, cache, table, pos, out=out, lse=lse)
    torch.cuda.synchronize()
    assert _lib.sync_status() == 0
    return out, lse


def _problem(D, dtype, M, n, std, seed=0, H=16, G=2):
    import torch

    g = torch.Generator(device="cuda").manual_seed(seed)
    cols = -(-n // 32)
    cache = make_cache(g, cols + 1, 32, G, D, dtype, 4)
    v = make_cache(g, cols + 1, 32, G, D, dtype, 4, std=std)
    cache.v.copy_(v.v)
    cache.v_scale.copy_(v.v_scale)
    table = torch.randperm(cols + 1, generator=g, device="cuda")[:cols].view(1, cols).int()
    pos = torch.arange(n - M, n, device="cuda").view(1, M).int()
    q = torch.randn((1, M, H, D), generator=g, device="cuda").to(dt(dtype))
    return q, cache, table, pos


def _set_row(cache, table, j, low, key=None):
    """Row j of the sequence: V constant; K a multiple of `key` [G, D / 2] codes."""
    page, off = table[0, j // cache.page_size], j % cache.page_size
    cache.v[page, off] = 0
    cache.v_scale[page, :, off, 0], cache.v_scale[page, :, off, 1] = 0, low
    if key is not None:
        cache.k[page, off] = 0
        cache.k_scale[page, :, off, 0], cache.k_scale[page, :, off, 1] = 0, key


@pytest.mark.parametrize("M", [1, 2, 20])
@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "bf16"), (64, "f16"), (128, "f16")])
@pytest.mark.parametrize("std,low", [(0.1, 0.0), (0.005, 0.0), (1e-4, 0.0), (1e-4, 1e-3), (1.0, 1e-3),
                                     (1e-4, -30.0)])
@pytest.mark.parametrize("weight", [0.3, 0.9, 0.98])
def test_a_constant_row_with_much_of_the_weight(weight, std, low, D, dtype, M):
    """One row, whose key is a constant that gives it about `weight` of the softmax."""
    import math

    import torch

    n = 500
    q, cache, table, pos = _problem(D, dtype, M, n, std)
    q = q.abs()  # so that one constant key does for every head
    for j in (3, 130):
        _set_row(cache, table, j, 0.0, -100.0 / D)  # (and some that nobody weighs)
    q *= 0.3
    mean = q.float().sum(-1).mean().item() / math.sqrt(D)  # of a key of ones
    _set_row(cache, table, 77, low, math.log(n * weight / (1 - weight)) / mean)
    out, lse = _attn(q, cache, table, pos)
    check_attn(q, cache, table, pos, -1, 0, None, out, lse, dtype)


@pytest.mark.parametrize("M", [1, 2, 20])
@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "bf16"), (64, "f16"), (128, "f16")])
@pytest.mark.parametrize("low", [0.0, 1e-3, -7.0, 1e30, -3e38])
@pytest.mark.parametrize("share", [0.5, 1.0])
def test_many_constant_rows(share, low, D, dtype, M):
    """Half of the rows, or all; where all are zero, O is zero."""
    import torch

    if dtype == "f16" and abs(low) > 1e4:
        low = 60000.0 if low > 0 else -60000.0
    q, cache, table, pos = _problem(D, dtype, M, 500, 0.02, 3)
    for j in range(500):
        if share == 1.0 or j % 2:
            _set_row(cache, table, j, low)
    out, lse = _attn(q, cache, table, pos)
    check_attn(q, cache, table, pos, -1, 0, None, out, lse, dtype)
    if share == 1.0 and low == 0.0:
        assert (out == 0).all()


@pytest.mark.parametrize("M", [1, 20])
def test_constant_rows_among_large_ones(M):
    """Zero rows beside rows whose steps are up to 2^40."""
    q, cache, table, pos = _problem(64, "bf16", M, 300, 2.0 ** 40, 5)
    for j in range(0, 300, 3):
        _set_row(cache, table, j, 0.0)
    out, lse = _attn(q, cache, table, pos)
    check_attn(q, cache, table, pos, -1, 0, None, out, lse, "bf16")
