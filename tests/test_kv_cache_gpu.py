"""nsa_kv_append and nsa_kv_read.

Q, and K before it is stored, are nsa_qk_norm_rope's bits (whose own tests hold
it to the float64 oracle); a 4-bit row is what the oracle makes of that 16-bit
row, code for code, but where (x - low) / step is within 2^-16 of the middle of
two codes (its fp32 rounding: x - low and the quotient, 2 x 2^-24 of 15). What
is read is low + step code rounded: half a unit of the 16-bit type, and 2^-23
for the fp32 sum before it.
"""

import numpy as np
import pytest

import oracle.norm_rope as R
import oracle.paged as P
from _paged import TINY, U, dt, make_cache, np64, rows_of
from _parity import poisoned

pytestmark = pytest.mark.gpu


def _inputs(B, M, H, G, D, dtype, rot, seed, fused=False, weights=True, rows=600):
    import torch

    from nsa_block_selection_gb300 import rope_tables

    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    if fused:
        x = (1.5 * rand(B, M, H + 2 * G, D)).to(dt(dtype))
        q, k, v = x[:, :, :H], x[:, :, H:H + G], x[:, :, H + G:]
    else:
        q, k, v = ((1.5 * rand(B, M, n, D)).to(dt(dtype)) for n in (H, G, G))
    wq, wk = ((1 + 0.3 * rand(D)) for _ in range(2)) if weights else (None, None)
    cos, sin = rope_tables(rows, rot) if rot else (None, None)
    return g, q, k, v, wq, wk, cos, sin


def _places(B, M, page, seed, pad=True, limit=600):
    """Distinct places: a run of positions for every sequence, some of them
    padding, some in pages that the sequence does not have."""
    import torch

    rng = np.random.default_rng(seed)
    cols = -(-limit // page)
    table = rng.permutation(B * cols + 3)[:B * cols].reshape(B, cols).astype(np.int32)
    pos = np.stack([rng.permutation(limit)[:M] for _ in range(B)]).astype(np.int32)
    if pad:
        pos[rng.random((B, M)) < 0.2] = -1
        table[rng.random((B, cols)) < 0.2] = -1
    return torch.from_numpy(table).cuda(), torch.from_numpy(pos).cuda(), B * cols + 3


def _bytes(cache):
    return [None if t is None else t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]


def _check_append(args, cache, table, pos, eps, inter, dtype):
    """Appends, and checks every byte of the cache and Q's rows."""
    import torch

    from nsa_block_selection_gb300 import kv_append, qk_norm_rope

    _, q, k, v, wq, wk, cos, sin = args
    before = _bytes(cache)
    q_out = poisoned(q.shape, q.dtype)
    got = kv_append(q, k, v, cache, table, pos, wq, wk, cos, sin, eps=eps, interleaved=inter,
                    q_out=q_out)
    torch.cuda.synchronize()
    assert got is q_out
    if eps is not None:
        wantq, wantk = qk_norm_rope(q, k, wq, wk, cos, sin, pos, eps=eps, interleaved=inter)
    else:  # (rotation alone: the oracle's, which has no norm at eps = 1 - mean(x^2))
        wantq, wantk = _rotated(q, cos, sin, pos, inter), _rotated(k, cos, sin, pos, inter)
    assert torch.equal(q_out.view(torch.int16), wantq.view(torch.int16))
    tn, pn = table.cpu().numpy(), pos.cpu().numpy()
    rows = cos.shape[0] if cos is not None else 1 << 30
    page = cache.page_size
    at = [(b, m, P.place(tn[b], int(pn[b, m]), page, cache.pages))
          for b in range(pn.shape[0]) for m in range(pn.shape[1]) if pn[b, m] < rows]
    at = [(b, m, *x) for b, m, x in at if x is not None]
    b, m, pg, off = (np.array(x, dtype=np.int64) for x in zip(*at))
    for name, src, was, was_scale in (("k", wantk, *before[0::2]), ("v", v, *before[1::2])):
        now, x = getattr(cache, name), src[b, m]
        if cache.bits == 16:
            want = was.clone()
            want[pg, off] = x
            assert torch.equal(now.view(torch.int16), want.view(torch.int16)), name
            continue
        scale = getattr(cache, name + "_scale")
        xf = np64(x)
        code, step, low = P.quantise(xf)
        s = np64(scale)[pg, :, off]
        assert (s[..., :1] == step).all() and (s[..., 1:] == low).all(), name
        c = now.cpu().numpy()[pg, off]
        c = np.stack([c & 15, c >> 4], -1).reshape(xf.shape)
        quot = (xf - low) / np.where(step > 0, step, 1)
        tie = np.abs(np.abs(quot - np.floor(quot)) - 0.5) < 2.0 ** -16
        assert ((c == code) | (tie & (np.abs(c - code) == 1))).all(), name
        keep, keep_scale = was.clone(), was_scale.clone()
        keep[pg, off] = now[pg, off]
        keep_scale[pg, :, off] = scale[pg, :, off]
        assert torch.equal(now, keep), f"{name}: other rows were written"
        assert torch.equal(scale.view(torch.int16), keep_scale.view(torch.int16)), name


def _rotated(x, cos, sin, pos, inter):
    """Rotation without a norm, in fp32 with the kernel's roundings (two
    products and a sum, which may be fused: compared through the oracle)."""
    import torch

    c, s = cos[pos.clamp(0).long()][:, :, None], sin[pos.clamp(0).long()][:, :, None]
    half = cos.shape[1]
    y = x.float().clone()
    a, b = (y[..., 0:2 * half:2], y[..., 1:2 * half:2]) if inter else (y[..., :half], y[..., half:2 * half])
    a, b = (a.double() * c - b.double() * s), (b.double() * c + a.double() * s)
    if inter:
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a.float(), b.float()
    else:
        y[..., :half], y[..., half:2 * half] = a.float(), b.float()
    y = y.to(x.dtype)
    return torch.where((pos >= 0)[:, :, None, None], y, torch.zeros_like(y))


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("D,dtype,H,G,rot,inter,page,fused", [
    (128, "bf16", 64, 8, 128, False, 64, True), (64, "f16", 16, 2, 32, True, 16, False),
    (64, "bf16", 1, 1, 64, False, 32, True), (128, "f16", 3, 3, 64, True, 128, False),
    (128, "bf16", 7, 1, 0, False, 16, True), (64, "f16", 2, 5, 16, False, 1024, True)])
@pytest.mark.parametrize("B,M", [(1, 1), (3, 77), (48, 1)])
def test_append(B, M, D, dtype, H, G, rot, inter, page, fused, bits):
    args = _inputs(B, M, H, G, D, dtype, rot, 10 * M + B, fused)
    table, pos, pages = _places(B, M, page, B + M)
    cache = make_cache(args[0], pages, page, G, D, dtype, bits)
    table[0, 0] = 0  # at least one token is stored
    pos[0, 0] = 3
    if M > 1:
        pos[0, 1:][pos[0, 1:] < page] = -1
    table[1:][table[1:] == 0] = -1
    table[0, 1:][table[0, 1:] == 0] = -1
    _check_append(args, cache, table, pos, 1e-6, inter, dtype)


@pytest.mark.parametrize("layout", ["joint", "heads"])
def test_append_strided_cache(layout):
    args = _inputs(2, 50, 8, 2, 128, "bf16", 128, 3, True)
    table, pos, pages = _places(2, 50, 32, 4)
    cache = make_cache(args[0], pages, 32, 2, 128, "bf16", 16, layout)
    assert not cache.k.is_contiguous()
    _check_append(args, cache, table, pos, 1e-6, False, "bf16")


@pytest.mark.parametrize("bits", [16, 4])
def test_append_positions_past_the_angle_tables_are_padding(bits):
    args = _inputs(2, 40, 4, 2, 64, "f16", 64, 5, rows=100)
    table, pos, pages = _places(2, 40, 16, 6, pad=False, limit=200)
    cache = make_cache(args[0], pages, 16, 2, 64, "f16", bits)
    assert (pos >= 100).any() and (pos < 100).any()
    _check_append(args, cache, table, pos, 1e-6, False, "f16")


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_without_norm(inter):
    """Against the float64 turn: the store's half unit, and fp32 products."""
    import torch

    from nsa_block_selection_gb300 import kv_append, kv_read

    g, q, k, v, _, _, cos, sin = _inputs(2, 30, 4, 2, 64, "bf16", 32, 8)
    table, pos, pages = _places(2, 30, 16, 9, pad=False)
    cache = make_cache(g, pages, 16, 2, 64, "bf16", 16)
    out = kv_append(q, k, v, cache, table, pos, cos=cos, sin=sin, eps=None, interleaved=inter)
    kk, vv = kv_read(cache, table, pos)
    assert torch.equal(vv, v)
    pn = pos.cpu().numpy()
    c, s = np64(cos)[pn][:, :, None], np64(sin)[pn][:, :, None]
    for got, x in ((out, q), (kk, k)):
        want = R.turn(np64(x), c, s, inter)
        mag = np.abs(R.turn(np.abs(np64(x)), np.abs(c), -np.abs(s), inter)) + np.abs(want)
        assert (np.abs(np64(got) - want) <= U["bf16"] * np.abs(want) + 4 * 2.0 ** -24 * mag
                + TINY["bf16"]).all()


@pytest.mark.parametrize("bits", [16, 4])
def test_keys_and_values_alone(bits):
    import torch

    from nsa_block_selection_gb300 import kv_append

    args = _inputs(2, 30, 4, 2, 64, "bf16", 64, 12, True)
    g, q, k, v, wq, wk, cos, sin = args
    table, pos, pages = _places(2, 30, 16, 13)
    a, b = (make_cache(torch.Generator(device="cuda").manual_seed(1), pages, 16, 2, 64, "bf16", bits)
            for _ in range(2))
    assert kv_append(None, k, v, a, table, pos, None, wk, cos, sin) is None
    kv_append(q, k, v, b, table, pos, wq, wk, cos, sin)
    for x, y in zip(_bytes(a), _bytes(b)):
        assert (x is None and y is None) or torch.equal(x, y)


def test_query_in_place_and_positions_of_a_prompt():
    """Q of a fused projection turned where it lies; positions None: 0 .. M - 1."""
    import torch

    from nsa_block_selection_gb300 import kv_append, kv_read, qk_norm_rope

    g, q, k, v, wq, wk, cos, sin = _inputs(2, 130, 8, 2, 128, "bf16", 128, 14, True)
    wantq, wantk = qk_norm_rope(q, k, wq, wk, cos, sin)
    keep = v.clone()
    table, _, pages = _places(2, 130, 64, 15, pad=False, limit=130)
    cache = make_cache(g, pages, 64, 2, 128, "bf16", 16)
    kv_append(q, k, v, cache, table, None, wq, wk, cos, sin, q_out=q)
    assert torch.equal(q, wantq) and torch.equal(v, keep)
    pos = torch.arange(130, device="cuda", dtype=torch.int32)
    kk, vv = kv_read(cache, table, pos)
    assert torch.equal(kk, wantk) and torch.equal(vv, keep)


def test_rows_that_four_bits_cannot_hold_plainly():
    """Constant rows, zeros, ranges too small for a step, one huge entry, the
    ends of the types, and rows that are not finite."""
    import torch

    from nsa_block_selection_gb300 import kv_append, kv_read

    x = torch.zeros((1, 12, 1, 64), device="cuda")
    x[0, 1] = 3.25
    x[0, 2] = -1e-30
    x[0, 3, 0, 5] = 2.0 ** -58  # step 2^-58 / 15 < 2^-60
    x[0, 4, 0, ::2], x[0, 4, 0, 1::2] = 1e30, -1e30
    x[0, 5, 0, 7] = float("inf")
    x[0, 6, 0, 9] = float("nan")
    x[0, 7, 0, 0], x[0, 7, 0, 1] = 3.3e38, -3.3e38  # wider than fp32
    x[0, 8] = torch.linspace(-1, 1, 64, device="cuda")
    x[0, 9] = 1.0
    x[0, 9, 0, 63] = -float("inf")
    x[0, 10, 0, 1] = -0.0
    x[0, 11] = torch.linspace(100, 101, 64, device="cuda")
    v = x.bfloat16()
    g = torch.Generator(device="cuda").manual_seed(0)
    cache = make_cache(g, 1, 16, 1, 64, "bf16", 4)
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    k = torch.randn((1, 12, 1, 64), generator=g, device="cuda").bfloat16()
    kv_append(None, k, v, cache, table)
    pos = torch.arange(12, device="cuda", dtype=torch.int32)
    _, got = kv_read(cache, table, pos)
    bad = [5, 6, 7, 9]
    assert torch.isnan(got[0, bad]).all()
    fine = [i for i in range(12) if i not in bad]
    code, step, low = P.quantise(np64(v[0, fine]))
    want = low + step * code
    assert (np.abs(np64(got[0, fine]) - want) <= U["bf16"] * (1 + 2.0 ** -10) * np.abs(want)
            + TINY["bf16"]).all()
    assert (got[0, [0, 1, 2, 10]] == v[0, [0, 1, 2, 10]]).all()


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("G,D,dtype,page,layout", [(1, 64, "f16", 16, "plain"), (8, 128, "bf16", 64, "plain"),
                                                   (3, 128, "f16", 32, "joint"), (2, 64, "bf16", 256, "heads")])
def test_read(G, D, dtype, page, layout, bits):
    import torch

    from nsa_block_selection_gb300 import kv_read

    table, pos, pages = _places(3, 200, page, G)
    pos[0, 0], pos[0, 1] = 2 ** 31 - 1, table.shape[1] * page  # past the table
    g = torch.Generator(device="cuda").manual_seed(G)
    cache = make_cache(g, pages, page, G, D, dtype, bits, layout)
    for out in ([dtype] if bits == 16 else ["f16", "bf16"]):
        shape = (3, 200, G, D)
        k, v = kv_read(cache, table, pos, dtype=dt(out), k_out=poisoned(shape, dt(out)),
                       v_out=poisoned(shape, dt(out)))
        tn, pn = table.cpu().numpy(), pos.cpu().numpy()
        for got, name in ((k, "k"), (v, "v")):
            rows = rows_of(cache, name)[0]
            want = np.zeros(shape)
            for b in range(3):
                for m in range(200):
                    at = P.place(tn[b], int(pn[b, m]), page, pages)
                    if at is not None:
                        want[b, m] = rows[at]
            slack = 0 if bits == 16 else U[out] * (1 + 2.0 ** -10) * np.abs(want) + TINY[out]
            assert (np.abs(np64(got) - want) <= slack).all()
