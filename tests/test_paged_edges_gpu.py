"""Calls of the paged cache at the ends of what is allowed: rows that may hold
anything under every kind of row tile, positions in any order, twice, or past the
page table, pages that sequences share, the largest table, empty batches.
"""

import numpy as np
import pytest

from _paged import check_attn, make_cache
from _parity import poisoned

pytestmark = pytest.mark.gpu

BITS = [16, 4]
FAR = 2 ** 31 - 32  # the last position


def _attn(q, cache, table, pos, left=-1, sinks=0):
    import torch

    from nsa_block_selection_gb300 import _lib, paged_attn

    B, M, H, D = q.shape
    out = paged_attn(q, cache, table, pos, window=(left, 0), sinks=sinks, out=poisoned(q.shape, q.dtype),
                     lse=poisoned((B, H, M), torch.float32))
    torch.cuda.synchronize()
    assert _lib.sync_status() == 0
    return out


def _case(B, M, H, G, D, dtype, bits, page, cols, seed, std=1.0):
    import torch

    from _paged import dt

    g = torch.Generator(device="cuda").manual_seed(seed)
    cache = make_cache(g, B * cols, page, G, D, dtype, bits, std=std)
    table = torch.randperm(B * cols, generator=g, device="cuda").view(B, cols).int()
    q = torch.randn((B, M, H, D), generator=g, device="cuda").to(dt(dtype))
    return q, cache, table


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("M", [4, 8, 20, 45])  # rows of a KV head: 16, 32, 80, 180
@pytest.mark.parametrize("page,D,dtype", [(16, 64, "f16"), (256, 128, "bf16")])
def test_rows_that_nobody_sees(M, page, D, dtype, bits):
    import torch

    n, left, sinks = 530, 40, 5
    cols = -(-n // page) + 1
    q, cache, table = _case(2, M, 8, 2, D, dtype, bits, page, cols, 50 + M)
    pos = torch.tensor([list(range(n - M, n)), [-1] * M], dtype=torch.int32, device="cuda")
    clean = _attn(q, cache, table, pos, left, sinks)
    seen = torch.zeros((2 * cols, page), dtype=torch.bool, device="cuda")
    for j in range(n):
        if j >= n - M - left or j < sinks:
            seen[table[0, j // page], j % page] = True
    if bits == 16:
        cache.k[~seen], cache.v[~seen] = float("nan"), float("inf")
    else:
        cache.k_scale.transpose(1, 2)[~seen] = float("nan")
        cache.v_scale.transpose(1, 2)[~seen] = float("inf")
    q[1] = float("nan")
    got = _attn(q, cache, table, pos, left, sinks)
    for x, y in zip(clean, got):
        assert torch.equal(x[:1], y[:1])
    assert (got[0][1] == 0).all() and (got[1][1] == -float("inf")).all()


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("M", [3, 20])
def test_queries_that_are_not_finite_stay_in_their_row(M, bits):
    import torch

    q, cache, table = _case(1, M, 4, 1, 64, "bf16", bits, 32, 10, 61)
    pos = torch.arange(300 - M, 300, dtype=torch.int32, device="cuda")
    want = _attn(q, cache, table, pos)
    q[0, 1, 1, 3] = float("nan")
    got = _attn(q, cache, table, pos)
    bad = torch.zeros((1, M, 4), dtype=torch.bool, device="cuda")
    bad[0, 1, 1] = True
    assert torch.isnan(got[0][bad]).all() and torch.isnan(got[1].transpose(1, 2)[bad]).all()
    assert torch.equal(got[0][~bad], want[0][~bad])
    assert torch.equal(got[1].transpose(1, 2)[~bad], want[1].transpose(1, 2)[~bad])


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("M,H,G", [(7, 2, 2), (7, 4, 2), (24, 8, 2)])
@pytest.mark.parametrize("left,sinks", [(-1, 0), (33, 3)])
def test_positions_in_any_order_and_twice(M, H, G, left, sinks, bits):
    """Also one past the table, whose window lies behind its end."""
    import torch

    q, cache, table = _case(3, M, H, G, 64, "f16", bits, 16, 20, 71)
    pos = torch.randint(0, 320, (3, M), generator=torch.Generator().manual_seed(5)).int()
    pos[0, 1] = pos[0, 0]
    pos[1, 2:5] = torch.tensor([-1, 5000, 319])
    pos[2, 0], pos[2, M - 1] = FAR, 0
    table[1] = table[0]  # pages that two sequences share
    pos = pos.cuda()
    out, lse = _attn(q, cache, table, pos, left, sinks)
    check_attn(q, cache, table, pos, left, sinks, None, out, lse, "f16")


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("M,H", [(1, 4), (3, 4), (20, 4)])
def test_the_largest_table(M, H, bits):
    """2^30 tokens, of which a sequence has its first and last page: the same as
    those two alone."""
    import torch

    page, cols = 1024, 2 ** 20
    q, cache, two = _case(1, M, H, 1, 64, "f16", bits, page, 2, 81)
    table = torch.full((1, cols), -1, dtype=torch.int32, device="cuda")
    table[0, 0], table[0, -1] = two[0, 0], two[0, 1]
    near = torch.arange(2 * page - M, 2 * page, dtype=torch.int32, device="cuda")
    out, lse = _attn(q, cache, table, near + (cols - 2) * page)
    check_attn(q, cache, two, near, -1, 0, None, out, lse, "f16")
    out, lse = _attn(q, cache, table, near + (cols - 2) * page, 500, 40)
    check_attn(q, cache, two, near, 500, 40, None, out, lse, "f16")


@pytest.mark.parametrize("bits", BITS)
def test_positions_at_the_end_of_the_type(bits):
    """A window of every key from the last position on; a cache that ends long before."""
    import torch

    for M in (1, 20):
        q, cache, table = _case(1, M, 4, 2, 64, "f16", bits, 16, 3, 91)
        pos = torch.full((1, M), FAR, dtype=torch.int32, device="cuda")
        for left, sinks in ((-1, 0), (2 ** 40, 0), (FAR - 20, 0), (0, 2 ** 40)):
            out, lse = _attn(q, cache, table, pos, left, sinks)
            check_attn(q, cache, table, pos, left, sinks, None, out, lse, "f16")


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("B,M", [(0, 1), (2, 0), (0, 0)])
def test_nothing_to_do(B, M, bits):
    import torch

    import nsa_block_selection_gb300 as nsa

    _, cache, _ = _case(1, 1, 4, 2, 64, "f16", bits, 16, 3, 95)
    before = [t.clone() for t in (cache.k, cache.v)]
    q = torch.zeros((B, M, 4, 64), dtype=torch.float16, device="cuda")
    kv = torch.zeros((B, M, 2, 64), dtype=torch.float16, device="cuda")
    table = torch.zeros((B, 3), dtype=torch.int32, device="cuda")
    pos = torch.zeros((B, M), dtype=torch.int32, device="cuda")
    assert nsa.kv_append(q, kv, kv, cache, table, pos).shape == q.shape
    assert nsa.kv_append(None, kv, kv, cache, table, pos, eps=None) is None
    o, lse = nsa.paged_attn(q, cache, table, pos)
    assert o.shape == q.shape and lse.shape == (B, 4, M)
    k, v = nsa.kv_read(cache, table, pos, dtype=torch.float16)
    assert k.shape == v.shape == kv.shape
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(before, (cache.k, cache.v)))


@pytest.mark.parametrize("bits", BITS)
def test_append_writes_no_other_row(bits):
    """One token in each of two sequences of a padded batch: every byte of the cache
    beside their rows stays, for both forms of the kernel."""
    import torch

    import nsa_block_selection_gb300 as nsa

    for H, G in ((4, 2), (64, 8)):
        q, cache, table = _case(3, 40, H, G, 128, "bf16", bits, 16, 4, 97)
        x = torch.randn((3, 40, 2, G, 128), device="cuda").bfloat16()
        pos = torch.full((3, 40), -1, dtype=torch.int32, device="cuda")
        pos[0, 39], pos[2, 0] = 63, 17
        table[1] = -1
        parts = [t for t in (cache.k, cache.v, cache.k_scale, cache.v_scale) if t is not None]
        before = [t.clone() for t in parts]
        nsa.kv_append(q, x[:, :, 0], x[:, :, 1], cache, table, pos)
        torch.cuda.synchronize()
        for i, (t, b) in enumerate(zip(parts, before)):
            diff = (t.view(torch.uint8) != b.view(torch.uint8)).flatten(2).any(2) if i < 2 else \
                (t.view(torch.int16) != b.view(torch.int16)).any(3).any(1)
            want = torch.zeros_like(diff)
            want[table[0, 3], 15] = want[table[2, 1], 1] = True
            assert torch.equal(diff, want)


@pytest.mark.parametrize("M,H,G,D,dtype,bits,B", [
    (20, 16, 8, 64, "f16", 16, 24), (20, 32, 8, 128, "bf16", 4, 24), (1, 16, 8, 128, "bf16", 16, 48),
    (3, 24, 8, 64, "f16", 16, 48), (1, 16, 16, 128, "f16", 4, 70), (2, 32, 32, 64, "bf16", 4, 90)])
def test_more_items_than_shares_and_empty_ones(M, H, G, D, dtype, bits, B):
    """Cut items among many: padding sequences between them, sequences that share pages."""
    import torch

    from _paged import dt

    g = torch.Generator(device="cuda").manual_seed(99 + B)
    rng = np.random.default_rng(99 + B)
    cache = make_cache(g, 48, 64, G, D, dtype, bits)
    table = torch.from_numpy(rng.integers(0, 48, (B, 40)).astype(np.int32)).cuda()
    lens = rng.integers(M, 2560, B)
    pos = np.stack([np.arange(n - M, n) for n in lens]).astype(np.int32)
    pos[::5] = -1
    pos[3, M // 2:] = -1
    pos[-1] = -7
    q = torch.randn((B, M, H, D), generator=g, device="cuda").to(dt(dtype))
    pos = torch.from_numpy(pos).cuda()
    out, lse = _attn(q, cache, table, pos)
    some = [0, 1, 3, 4, B // 2, B - 3, B - 2, B - 1]
    check_attn(q[some], cache, table[some], pos[some], -1, 0, None, out[some], lse[some], dtype)
    empty = (pos < 0)
    assert (out[empty] == 0).all() and (lse.transpose(1, 2)[empty] == -float("inf")).all()
    # each sequence by itself, in other shares: the roundings of p are independent, so in
    # norm each result is off by the two roundings (p's and O's) of at most u each; twice
    for b in range(B):
        o, _ = _attn(q[b:b + 1], cache, table[b:b + 1], pos[b:b + 1])
        u = torch.finfo(o.dtype).eps / 2
        far = (o.double() - out[b:b + 1].double()).norm()
        assert far <= 8 * u * o.double().norm() + 1e-30, (b, far)
