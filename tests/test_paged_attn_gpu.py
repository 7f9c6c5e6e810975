"""nsa_paged_attn against the float64 oracle (bounds: _paged.py)."""

import numpy as np
import pytest

from _paged import check_attn, dt, make_cache
from _parity import poisoned

pytestmark = pytest.mark.gpu


def _problem(B, M, H, G, D, dtype, bits, page, lens, seed, layout="plain", holes=0, std=1.0):
    """Sequences of `lens` tokens, the last M of them new; pages in random
    order, `holes` of each sequence's own taken away."""
    import torch

    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    cols = max(1, -(-max(lens) // page))
    cache = make_cache(g, B * cols + 2, page, G, D, dtype, bits, layout, std=std)
    table = rng.permutation(B * cols + 2)[:B * cols].reshape(B, cols).astype(np.int32)
    pos = np.full((B, M), -1, np.int32)
    for b, n in enumerate(lens):
        new = min(M, n)
        pos[b, :new] = np.arange(n - new, n)
        table[b, -(-n // page):] = -1
        for _ in range(holes):
            table[b, rng.integers(0, cols)] = rng.choice([-1, B * cols + 2, 2 ** 31 - 1])
    q = torch.randn((B, M, H, D), generator=g, device="cuda").to(dt(dtype))
    return q, cache, torch.from_numpy(table).cuda(), torch.from_numpy(pos).cuda()


def _run(q, cache, table, pos, left, sinks, dtype, scale=None, **kw):
    import torch

    from nsa_block_selection_gb300 import _lib, paged_attn

    B, M, H, D = q.shape
    out, lse = poisoned((B, M, H, D), q.dtype), poisoned((B, H, M), torch.float32)
    paged_attn(q, cache, table, pos, window=(left, 0), sinks=sinks, scale=scale, out=out, lse=lse,
               **kw)
    torch.cuda.synchronize()
    assert _lib.sync_status() == 0
    return out, lse


def _check(case, left, sinks, dtype, scale=None):
    out, lse = _run(*case, left, sinks, dtype, scale)
    q, cache, table, pos = case
    check_attn(q, cache, table, pos, left, sinks, scale, out, lse, dtype)


BITS = [16, 4]


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("D,dtype", [(64, "f16"), (128, "bf16"), (64, "bf16"), (128, "f16")])
@pytest.mark.parametrize("n", [1, 15, 16, 17, 33, 300])
def test_one_token_of_one_sequence(n, D, dtype, bits):
    _check(_problem(1, 1, 8, 2, D, dtype, bits, 16, [n], 100 + n), -1, 0, dtype)


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("H,G", [(1, 1), (2, 1), (3, 1), (7, 1), (8, 1), (9, 1), (16, 1), (24, 2),
                                 (10, 5), (4, 4)])
def test_heads(H, G, bits):
    _check(_problem(2, 2, H, G, 64, "f16", bits, 32, [70, 45], H * 10 + G), -1, 0, "f16")


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("left,sinks", [(-1, 0), (0, 0), (0, 3), (1, 0), (16, 0), (37, 4), (100, 16),
                                        (100, 17), (64, 300), (5000, 2), (-1, 9), (250, 0)])
@pytest.mark.parametrize("D,dtype", [(128, "bf16"), (64, "f16")])
def test_windows_and_first_tokens(left, sinks, D, dtype, bits):
    case = _problem(3, 3, 8, 2, D, dtype, bits, 16, [401, 290, 2], 7 + left + sinks)
    _check(case, left, sinks, dtype)


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("page", [16, 64, 256, 1024])
def test_page_sizes_and_missing_pages(page, bits):
    case = _problem(4, 2, 8, 2, 128, "bf16", bits, page, [1500, 1023, 64, 1], 3, holes=1)
    _check(case, -1, 0, "bf16")
    _check(case, 200, 20, "bf16")


@pytest.mark.parametrize("bits", BITS)
def test_no_page_at_all_and_padding(bits):
    q, cache, table, pos = _problem(3, 4, 4, 2, 64, "f16", bits, 16, [50, 3, 40], 5)
    table[2] = -1
    pos[0, 1] = -5  # padding between tokens
    out, lse = _run(q, cache, table, pos, -1, 0, "f16")
    assert (out[2] == 0).all() and (lse[2] == -float("inf")).all()
    assert (out[0, 1] == 0).all() and (out[1, 3] == 0).all() and (lse[0, :, 1] == -float("inf")).all()
    check_attn(q, cache, table, pos, -1, 0, None, out, lse, "f16")


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("M,H,G,lens,left,sinks", [
    (5, 16, 2, [2047, 900, 5, 1333], -1, 0), (65, 32, 4, [700, 65], 256, 16),
    (130, 4, 4, [130, 200], -1, 0), (33, 3, 1, [33, 400], 40, 5)])
def test_several_tokens(M, H, G, lens, left, sinks, bits):
    case = _problem(len(lens), M, H, G, 64, "f16", bits, 16, lens, M + H)
    _check(case, left, sinks, "f16")


@pytest.mark.parametrize("bits", BITS)
def test_long_sequences_are_cut(bits):
    """Shares that cut items, begin and end inside them, with empty ones between."""
    case = _problem(5, 1, 8, 1, 128, "bf16", bits, 64, [9000, 1, 4111, 64, 6500], 11)
    case[3][3] = -1
    _check(case, -1, 0, "bf16")


@pytest.mark.parametrize("bits", BITS)
def test_more_row_tiles_than_are_cut(bits):
    import torch

    from nsa_block_selection_gb300 import _lib

    B, M = 520, 1
    q, cache, table, pos = _problem(2, M, 16, 1, 64, "f16", bits, 16, [90, 33], 21)
    assert _lib.paged_attn_workspace_bytes(B, M, 16, 1, 64, 4096) == 0
    assert _lib.paged_attn_workspace_bytes(2, M, 16, 1, 64, 4096) > 0
    few = _run(q, cache, table, pos, -1, 0, "f16")
    at = torch.arange(B, device="cuda") % 2
    many = _run(q[at].contiguous(), cache, table[at].contiguous(), pos[at].contiguous(), -1, 0, "f16")
    check_attn(q, cache, table, pos, -1, 0, None, many[0][:2], many[1][:2], "f16")
    check_attn(q, cache, table, pos, -1, 0, None, *few, "f16")
    for x in many:
        assert torch.equal(x[0::2], x[:1].expand_as(x[0::2]))
        assert torch.equal(x[1::2], x[1:2].expand_as(x[1::2]))


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("D,dtype", [(64, "f16"), (128, "bf16")])
@pytest.mark.parametrize("M,H,G,page,lens,left,sinks", [
    (3, 8, 1, 16, [3, 300], -1, 0), (17, 1, 1, 32, [17, 18, 700], -1, 0), (16, 8, 1, 64, [129], -1, 0),
    (40, 14, 2, 128, [40, 1000], 100, 7), (130, 3, 3, 256, [513, 131], 0, 1), (200, 16, 2, 1024, [1300], -1, 0),
    (33, 10, 2, 16, [900, 333], 257, 130), (5, 100, 1, 64, [640, 5], -1, 0), (20, 130, 1, 64, [70], -1, 0)])
def test_many_rows(M, H, G, page, lens, left, sinks, D, dtype, bits):
    """Row tiles of the tensor cores: heads that 128 rows do not divide by, pages
    that a step of 128 keys holds several of, steps that are seen in part."""
    case = _problem(len(lens), M, H, G, D, dtype, bits, page, lens, M + H + page)
    _check(case, left, sinks, dtype)


@pytest.mark.parametrize("bits", BITS)
def test_many_rows_missing_pages_and_padding(bits):
    q, cache, table, pos = _problem(4, 24, 8, 2, 128, "bf16", bits, 32, [2500, 24, 400, 999], 31, holes=9)
    pos[0, 5:9] = -1
    pos[1] = -3
    table[2, 4:] = -1
    out, lse = _run(q, cache, table, pos, -1, 0, "bf16")
    assert (out[1] == 0).all() and (lse[1] == -float("inf")).all() and (out[0, 5:9] == 0).all()
    check_attn(q, cache, table, pos, -1, 0, None, out, lse, "bf16")
    _check((q, cache, table, pos), 300, 40, "bf16")


@pytest.mark.parametrize("bits", BITS)
def test_many_rows_long_and_cut(bits):
    case = _problem(3, 20, 16, 2, 64, "f16", bits, 64, [9000, 21, 5000], 33)
    _check(case, -1, 0, "f16")
    _check(case, 2000, 4, "f16")


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("M", [1, 2, 6])
def test_strided_queries_and_positions_of_a_batch(M, bits):
    import torch

    q, cache, table, pos = _problem(3, M, 16, 2, 64, "f16", bits, 16, [200, 200, 200], 35)
    x = torch.randn((3, M, 24, 64), device="cuda").half()
    x[:, :, 4:20] = q
    view = x[:, :, 4:20]
    assert not view.is_contiguous()
    one = pos[0].contiguous()
    a, b = _run(q, cache, table, pos, -1, 0, "f16"), _run(view, cache, table, one, -1, 0, "f16")
    for s, t in zip(a, b):
        assert torch.equal(s, t)


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("B,M,H,G,n", [(50, 5, 32, 8, 100), (90, 3, 16, 2, 700), (6, 18, 16, 16, 3500)])
def test_many_items_for_a_cta(B, M, H, G, n, bits):
    """More items than SMs, whole and cut: every CTA goes through several; the
    same sequence twice gives the same bits."""
    import torch

    half = _problem(B // 2, M, H, G, 64, "f16", bits, 64, [n - 7 * b % n + M for b in range(B // 2)], 37)
    q, cache, table, pos = half
    two = torch.cat((torch.arange(B // 2), torch.arange(B // 2))).cuda()
    out, lse = _run(q[two].contiguous(), cache, table[two].contiguous(), pos[two].contiguous(), -1, 0, "f16")
    some = slice(0, min(B // 2, 6))
    check_attn(q[some], cache, table[some], pos[some], -1, 0, None, out[some], lse[some], "f16")
    few = _run(*(x[some].contiguous() if x is not cache else x for x in half), -1, 0, "f16")
    check_attn(q[some], cache, table[some], pos[some], -1, 0, None, *few, "f16")
