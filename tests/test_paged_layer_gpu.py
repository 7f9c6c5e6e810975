"""The paged-cache calls together, as a layer that answers runs them, and where
they are run: graphs, streams, far offsets, rows that hold anything.
"""

import numpy as np
import pytest

import oracle.paged as P
from _paged import U, check_attn, dt, make_cache, np64, rows_of
from _parity import poisoned

pytestmark = pytest.mark.gpu


def _sync():
    import torch

    from nsa_block_selection_gb300 import _lib

    torch.cuda.synchronize()
    assert _lib.sync_status() == 0


def _layer(x, H, G, w, tables, cache, table, pos, window, sinks, **kw):
    """Norm, rotation and cache, then attention: x [B, M, H + 2G, D]."""
    from nsa_block_selection_gb300 import kv_append, paged_attn

    q = kv_append(x[:, :, :H], x[:, :, H:H + G], x[:, :, H + G:], cache, table, pos, *w, *tables)
    return q, *paged_attn(q, cache, table, pos, window=window, sinks=sinks, **kw)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("window,sinks", [((-1, 0), 0), ((20, 0), 3)])
def test_prompt_then_tokens(window, sinks, bits):
    """A prompt of two sequences, padded, then drafted tokens and single ones:
    every output against the oracle on what the cache holds, and (16 bits,
    without first tokens) against the sliding-window forward of the whole."""
    import torch

    from nsa_block_selection_gb300 import kv_cache, kv_read, qk_norm_rope, rope_tables, swa_fwd

    g = torch.Generator(device="cuda").manual_seed(3)
    B, H, G, D, n = 2, 8, 2, 64, 60
    x = torch.randn((B, n, H + 2 * G, D), generator=g, device="cuda").bfloat16()
    w = [1 + 0.2 * torch.randn(D, generator=g, device="cuda") for _ in range(2)]
    tables = rope_tables(128, D)
    cache = kv_cache(20, 16, G, D, bits=bits)
    table = torch.randperm(20, generator=g, device="cuda")[:2 * 8].view(2, 8).int()
    lens, got, qs = [37, 44], [[], []], [[], []]
    steps = [44] + [3, 3] + [1] * 4
    at = [0, 0]
    for m in steps:
        pos = torch.full((B, m), -1, dtype=torch.int32)
        xs = torch.full((B, m, H + 2 * G, D), float("nan"))
        for b in range(B):
            new = min(m, lens[b]) if m == 44 else m
            pos[b, :new] = torch.arange(at[b], at[b] + new)
            xs[b, :new] = x[b, at[b]:at[b] + new].float().cpu()
            at[b] += new
        pos, xs = pos.cuda(), xs.cuda().bfloat16()
        q, o, lse = _layer(xs, H, G, w, tables, cache, table, pos, window, sinks)
        _sync()
        check_attn(q, cache, table, pos, window[0], sinks, None, o, lse, "bf16")
        for b in range(B):
            live = (pos[b] >= 0)
            got[b].append(o[b][live])
            qs[b].append(q[b][live])
            assert (o[b][~live] == 0).all()
    for b in range(B):
        o, q = torch.cat(got[b])[None], torch.cat(qs[b])[None]
        L = o.shape[1]
        wq, wk = qk_norm_rope(x[b:b + 1, :L, :H], x[b:b + 1, :L, H:H + G], *w, *tables)
        assert torch.equal(q, wq)
        pos = torch.arange(L, dtype=torch.int32, device="cuda")
        kk, vv = kv_read(cache, table[b:b + 1].contiguous(), pos)
        if bits == 16:
            assert torch.equal(kk, wk) and torch.equal(vv, x[b:b + 1, :L, H + G:])
        if sinks == 0:  # both round p, and O: twice the bound of one
            want, _ = swa_fwd(wq, kk, vv.contiguous(), window=window)
            mag = vv.float().abs().max().item()
            # (4 bits: what is read is rounded to 16 bits: u of k in the scores, and of v)
            slack = 4 * U["bf16"] * mag if bits == 16 else 16 * U["bf16"] * mag
            assert (o.float() - want.float()).abs().max().item() <= slack


def test_cached_rows_serve_the_selection_attention():
    import torch

    from nsa_block_selection_gb300 import kv_append, kv_cache, kv_read, sel_attn_fwd, topk_blocks

    g = torch.Generator(device="cuda").manual_seed(5)
    B, M, H, G, D = 1, 256, 16, 2, 128
    q, k, v = (torch.randn((B, M, n, D), generator=g, device="cuda").half() for n in (H, G, G))
    cache = kv_cache(8, 64, G, D, dtype=torch.float16)
    table = torch.tensor([[5, 0, 7, 2]], dtype=torch.int32, device="cuda")
    kv_append(None, k, v, cache, table, eps=None)
    kk, vv = kv_read(cache, table, torch.arange(M, dtype=torch.int32, device="cuda"))
    idx = topk_blocks(torch.randn((B, M, G, 4), generator=g, device="cuda"), M, 64, 3, 1, 1)
    for x, y in zip(sel_attn_fwd(q, kk, vv, idx, 64), sel_attn_fwd(q, k, v, idx, 64)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("bits", [16, 4])
def test_captured_steps(bits):
    """Decoding steps replayed from a graph with new inputs, positions and pages
    in place; the same bits as called."""
    import torch

    from nsa_block_selection_gb300 import rope_tables

    g = torch.Generator(device="cuda").manual_seed(8)
    B, H, G, D, page = 3, 16, 2, 128, 64
    tables = rope_tables(4096, D)
    a, b = (make_cache(torch.Generator(device="cuda").manual_seed(1), 200, page, G, D, "bf16", bits)
            for _ in range(2))
    table = torch.randperm(200, generator=g, device="cuda")[:B * 60].view(B, 60).int()
    x = torch.zeros((B, 1, H + 2 * G, D), device="cuda").bfloat16()
    pos = torch.zeros((B, 1), dtype=torch.int32, device="cuda")
    w = (None, None)
    _layer(x, H, G, w, tables, a, table, pos, (-1, 0), 0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _layer(x, H, G, w, tables, a, table, pos, (-1, 0), 0)
    for step in range(4):
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        pos.copy_(torch.tensor([[3000 + step], [5 * step], [700]]))
        if step == 2:
            table[1] = table[1].flip(0)
        graph.replay()
        if step == 0:  # the caches started alike, but for the capture's first call
            for s, t in zip((a.k, a.v, a.k_scale, a.v_scale), (b.k, b.v, b.k_scale, b.v_scale)):
                if s is not None:
                    t.copy_(s)
        want = _layer(x, H, G, w, tables, b, table, pos, (-1, 0), 0)
        _sync()
        for s, t in zip(out, want):
            assert torch.equal(s, t)


@pytest.mark.parametrize("bits", [16, 4])
def test_graphs_that_share_a_workspace(bits):
    import torch

    from nsa_block_selection_gb300 import _lib, paged_attn

    g = torch.Generator(device="cuda").manual_seed(9)
    ws = torch.empty(_lib.paged_attn_workspace_bytes(2, 1, 8, 1, 64, 4096), dtype=torch.uint8,
                     device="cuda").fill_(255)
    runs = []
    for n in (4000, 900):
        cache = make_cache(g, 140, 64, 1, 64, "f16", bits)
        table = torch.randperm(140, generator=g, device="cuda")[:128].view(2, 64).int()
        pos = torch.tensor([[n], [n // 3]], dtype=torch.int32, device="cuda")
        q = torch.randn((2, 1, 8, 64), generator=g, device="cuda").half()
        want = paged_attn(q, cache, table, pos)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = paged_attn(q, cache, table, pos, workspace=ws)
        runs.append((graph, out, want, cache, table, pos, q))
    for _ in range(3):
        for graph, *_ in runs:
            graph.replay()
    _sync()
    for _, out, want, *_ in runs:
        for s, t in zip(out, want):
            assert torch.equal(s, t)


@pytest.mark.parametrize("bits", [16, 4])
def test_side_streams_and_equal_bits(bits):
    """Calls that overlap on two streams, each with a workspace of its own, give
    the bits of calls one after another."""
    import torch

    from nsa_block_selection_gb300 import kv_append, kv_read, paged_attn

    g = torch.Generator(device="cuda").manual_seed(10)
    cache = make_cache(g, 600, 64, 4, 128, "bf16", bits)
    table = torch.randperm(600, generator=g, device="cuda")[:512].view(4, 128).int()
    pos = torch.tensor([[8000], [17], [4444], [8191]], dtype=torch.int32, device="cuda")
    q = torch.randn((4, 1, 32, 128), generator=g, device="cuda").bfloat16()
    want = paged_attn(q, cache, table, pos, sinks=2)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [paged_attn(q, cache, table, pos, sinks=2, stream=s) for _ in range(6) for s in streams]
    _sync()
    for out in outs:
        assert all(torch.equal(x, y) for x, y in zip(out, want))
    k, v = (torch.randn((4, 1, 4, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
    s = streams[0]
    got = kv_append(q, k, v, cache, table, pos, stream=s)
    rk, rv = kv_read(cache, table, pos, stream=s)
    s.synchronize()
    assert got.shape == q.shape
    if bits == 16:
        assert torch.equal(rv, v)
    assert kv_append(None, k, v, cache, table, pos, stream=s) is None
    other = type("S", (), {"device": torch.device("cuda:7")})()
    for call in (lambda: paged_attn(q, cache, table, pos, stream=other),
                 lambda: kv_read(cache, table, pos, stream=other),
                 lambda: kv_append(q, k, v, cache, table, pos, stream=other)):
        with pytest.raises(ValueError, match="stream"):
            call()
    _sync()


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("M", [1, 3])
def test_rows_that_nobody_sees_may_hold_anything(M, bits):
    """NaN and infinities after the last token of a page, in pages of others, behind
    the window and in padding queries."""
    import torch

    g = torch.Generator(device="cuda").manual_seed(11)
    page, n = 32, 139
    q = torch.randn((2, M, 8, 64), generator=g, device="cuda").half()
    cache = make_cache(g, 16, page, 2, 64, "f16", bits)
    table = torch.tensor([[3, 9, 1, 7, 12], [0, 5, 8, 2, 14]], dtype=torch.int32, device="cuda")
    pos = torch.tensor([list(range(n - M, n)), [-1] * M], dtype=torch.int32, device="cuda")
    clean = _attn(q, cache, table, pos)
    seen = torch.zeros((16, page), dtype=torch.bool, device="cuda")
    for j in range(n):
        if j >= n - M - 40 or j < 5:
            seen[table[0, j // page], j % page] = True
    bad = float("nan")
    if bits == 16:
        for t, b in ((cache.k, bad), (cache.v, float("inf"))):
            t[~seen] = b
    else:
        for t, b in ((cache.k_scale, bad), (cache.v_scale, float("inf"))):
            t.transpose(1, 2)[~seen] = b
    q[1] = bad
    got = _attn(q, cache, table, pos)
    for x, y in zip(clean, got):
        assert torch.equal(x[:1], y[:1])
    assert (got[0][1] == 0).all() and (got[1][1] == -float("inf")).all()


def _attn(q, cache, table, pos, left=40, sinks=5):
    import torch

    from nsa_block_selection_gb300 import paged_attn

    B, M, H, D = q.shape
    out = paged_attn(q, cache, table, pos, window=(left, 0), sinks=sinks, out=poisoned(q.shape, q.dtype),
                     lse=poisoned((B, H, M), torch.float32))
    _sync()
    return out


def test_scores_that_are_not_finite_stay_in_their_row():
    import torch

    from nsa_block_selection_gb300 import paged_attn

    g = torch.Generator(device="cuda").manual_seed(12)
    for bits in (16, 4):
        cache = make_cache(g, 4, 16, 1, 64, "bf16", bits)
        table = torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4)
        pos = torch.tensor([60], dtype=torch.int32, device="cuda")
        q = torch.randn((1, 1, 4, 64), generator=g, device="cuda").bfloat16()
        want = paged_attn(q, cache, table, pos)[0]
        q[0, 0, 1, 3] = float("nan")
        got, lse = paged_attn(q, cache, table, pos)
        _sync()
        assert torch.isnan(got[0, 0, 1]).all() and torch.isnan(lse[0, 1]).all()
        assert torch.equal(got[0, 0, [0, 2, 3]], want[0, 0, [0, 2, 3]])


@pytest.mark.parametrize("scale", [1e-4, 1e4])
@pytest.mark.parametrize("bits", [16, 4])
def test_sizes_of_values(bits, scale):
    """Small and large keys, values and queries."""
    import torch

    g = torch.Generator(device="cuda").manual_seed(13)
    cache = make_cache(g, 12, 32, 2, 64, "bf16", bits, std=scale)
    table = torch.randperm(12, generator=g, device="cuda")[:10].view(1, 10).int()
    pos = torch.tensor([[299]], dtype=torch.int32, device="cuda")
    q = (torch.randn((1, 1, 8, 64), generator=g, device="cuda") / scale).bfloat16()
    out, lse = _attn(q, cache, table, pos, -1, 0)
    check_attn(q, cache, table, pos, -1, 0, None, out, lse, "bf16")


@pytest.mark.parametrize("M", [1, 2, 20])
def test_rows_without_a_step(M):
    """Constant rows of K and of V among the others, and only such."""
    import torch

    g = torch.Generator(device="cuda").manual_seed(16)
    for share in (0.3, 1.0):
        cache = make_cache(g, 8, 32, 2, 64, "f16", 4)
        for name in ("k", "v"):
            some = torch.rand((8, 32, 2), generator=g, device="cuda") < share
            getattr(cache, name)[some] = 0
            scale = getattr(cache, name + "_scale")
            scale[..., 0].masked_fill_(some.transpose(1, 2), 0.0)
        table = torch.randperm(8, generator=g, device="cuda")[:7].view(1, 7).int()
        pos = torch.arange(200 - M, 200, dtype=torch.int32, device="cuda").view(1, M)
        q = torch.randn((1, M, 16, 64), generator=g, device="cuda").half()
        out, lse = _attn(q, cache, table, pos, -1, 0)
        check_attn(q, cache, table, pos, -1, 0, None, out, lse, "f16")


@pytest.mark.parametrize("bits", [16, 4])
def test_flat_attention_over_many_keys(bits):
    """Zero queries: O is the mean of the values, far smaller than they are. Its
    relative error in norm: the store's u / sqrt(3) at most, and fp32 sums of n
    terms, each off by 2^-24 of a partial sum of some sqrt(n) values (8 where they
    are codes less their mean): sqrt(n) 2^-24 of sqrt(n), against O of 1 / sqrt(n)
    of the values' size: n 2^-23 in all, 2 such (O and l)."""
    import torch

    from nsa_block_selection_gb300 import paged_attn

    g = torch.Generator(device="cuda").manual_seed(14)
    n = 16384
    cache = make_cache(g, n // 64, 64, 1, 128, "f16", bits)
    table = torch.randperm(n // 64, generator=g, device="cuda").view(1, -1).int()
    pos = torch.tensor([n - 1], dtype=torch.int32, device="cuda")
    q = torch.zeros((1, 1, 8, 128), device="cuda").half()
    o, lse = paged_attn(q, cache, table, pos)
    _sync()
    want = rows_of(cache, "v")[0].reshape(n, 128).mean(0)
    err = np.linalg.norm(np64(o)[0, 0] - want, axis=-1) / np.linalg.norm(want)
    assert err.max() <= U["f16"] / np.sqrt(3) + 4 * n * 2.0 ** -23
    assert np.abs(np64(lse) - np.log(n)).max() <= 2.0 ** -20 * (1 + np.log(n))


@pytest.mark.parametrize("bits", [16, 4])
def test_offsets_past_32_bits(bits):
    """Pages beyond 2^32 bytes of K and of V (and 2^31 scales' bytes)."""
    import torch

    from nsa_block_selection_gb300 import kv_append, kv_cache, kv_read, paged_attn

    g = torch.Generator(device="cuda").manual_seed(15)
    G, D, page = 8, 128, 64
    row = G * D * 2 if bits == 16 else G * D // 2
    pages = (1 << 32) // (row * page) + 50
    big, small = kv_cache(pages, page, G, D, bits=bits), kv_cache(6, page, G, D, bits=bits)
    far = torch.tensor([[pages - 1, 0, pages - 7, pages // 2, pages - 2, 3]], dtype=torch.int32,
                       device="cuda")
    near = torch.arange(6, dtype=torch.int32, device="cuda").view(1, 6)
    n = 6 * page
    q, k, v = (torch.randn((1, n, h, D), generator=g, device="cuda").bfloat16() for h in (8, G, G))
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    outs = []
    for cache, table in ((big, far), (small, near)):
        qq = kv_append(q, k, v, cache, table, pos)
        last = pos[-2:].contiguous()
        outs.append((qq, *kv_read(cache, table, pos),
                     *paged_attn(qq[:, -2:].contiguous(), cache, table, last)))
    _sync()
    for x, y in zip(*outs):
        assert torch.equal(x, y)


def test_refusals_on_the_gpu():
    import torch

    from nsa_block_selection_gb300 import NsaError, kv_append, kv_cache, kv_read, paged_attn

    cache = kv_cache(4, 16, 2, 64)
    table = torch.zeros((1, 4), dtype=torch.int32, device="cuda")
    pos = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    q, k = (torch.zeros((1, 1, n, 64), device="cuda").bfloat16() for n in (4, 2))
    bad = [
        lambda: paged_attn(q.half(), cache, table, pos), lambda: paged_attn(q[..., :32], cache, table, pos),
        lambda: paged_attn(q, cache, table.long(), pos), lambda: paged_attn(q, cache, table[0], pos),
        lambda: paged_attn(q, cache, table, pos.long()), lambda: paged_attn(q, cache, table, pos[:, :0]),
        lambda: paged_attn(q, cache, table, None), lambda: paged_attn(q, cache, table, pos, window=(3, 1)),
        lambda: paged_attn(q, cache, table, pos, sinks=-1), lambda: paged_attn(q[:, :, :3], cache, table, pos),
        lambda: paged_attn(q, cache, table, pos, out=q.float()),
        lambda: paged_attn(q, cache, table, pos, lse=pos.float()),
        lambda: paged_attn(q.cpu(), cache, table, pos), lambda: paged_attn(q, cache, table.cpu(), pos),
        lambda: kv_append(q, k, k[:, :, :1], cache, table, pos), lambda: kv_append(q, k.half(), k, cache, table),
        lambda: kv_append(q, k[:, :, :1], k[:, :, :1], cache, table, pos),
        lambda: kv_append(q.half(), k.half(), k.half(), cache, table, pos),
        lambda: kv_append(q, k, k, cache, table, pos, eps=-1.0),
        lambda: kv_append(q, k, k, cache, table, pos, q_weight=torch.ones(64, device="cuda"), eps=None),
        lambda: kv_read(cache, table, pos, dtype=torch.float16), lambda: kv_read(cache, table, None),
        lambda: kv_read(cache, table, pos, k_out=k.half()),
        lambda: paged_attn(q, kv_cache(4, 8, 2, 64), table, pos),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((TypeError, ValueError, NsaError, AttributeError)):
            call()
            pytest.fail(f"call {i} was not refused")
    _sync()
