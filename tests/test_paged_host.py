"""Refusals, workspace sizes and empty problems of the paged-cache entry points
(no GPU: arguments are rejected before any CUDA call), and the oracle's pins."""

import ctypes

import numpy as np
import pytest

import oracle.paged as P
from nsa_block_selection_gb300 import _lib

FAKE = 4096  # a 16-byte aligned non-null address that is never dereferenced
GOOD = dict(B=2, M=3, H=16, G=2, D=128, R=128, rows=100, ps=3, cols=4, eps=1e-6, dtype=1, wdtype=2,
            left=-1, sinks=0, pages=10, page=64, bits=16)


@pytest.fixture(scope="module")
def lib():
    import os

    if not os.path.exists(_lib.LIB_PATH):
        from nsa_block_selection_gb300.build import build

        build()
    return _lib.load()


def _kv(a, p):
    st = (a["page"] * a["G"] * a["D"], a["G"] * a["D"], a["D"])
    st = a.get("cstr", st + st)
    return (ctypes.c_uint64 * 13)(*(p[n] or 0 for n in ("kp", "vp", "ks", "vs")), a["pages"],
                                  a["page"], *(x % (1 << 64) for x in st), a["bits"])


def _ptrs(ptrs):
    names = ("q", "k", "v", "qo", "kp", "vp", "ks", "vs", "table", "wq", "wk", "cos", "sin", "pos", "o",
             "lse", "ws")
    p = dict.fromkeys(names, FAKE)
    p.update(ptrs or {})
    return p


V = ctypes.c_void_p


def _append(lib, ptrs=None, strides=None, cache=True, **over):
    a, p = dict(GOOD, **over), _ptrs(ptrs)
    s = None if strides is None else (ctypes.c_int64 * 12)(*strides)
    kv = _kv(a, p)
    return lib.nsa_kv_append(V(p["q"]), V(p["k"]), V(p["v"]), V(p["qo"]), kv if cache else None,
                             V(p["table"]), V(p["wq"]), V(p["wk"]), V(p["cos"]), V(p["sin"]),
                             V(p["pos"]), a["B"], a["M"], a["H"], a["G"], a["D"], a["R"], a["rows"],
                             a["ps"], a["cols"], a["eps"], 0, a["dtype"], a["wdtype"], s, None)


def _read(lib, ptrs=None, cache=True, **over):
    a, p = dict(GOOD, **over), _ptrs(ptrs)
    kv = _kv(a, p)
    return lib.nsa_kv_read(kv if cache else None, V(p["table"]), V(p["pos"]), V(p["k"]), V(p["v"]),
                           a["B"], a["M"], a["G"], a["D"], a["ps"], a["cols"], a["dtype"], None)


def _attn(lib, ptrs=None, strides=None, cache=True, ws_bytes=1 << 30, **over):
    a, p = dict(GOOD, **over), _ptrs(ptrs)
    s = None if strides is None else (ctypes.c_int64 * 3)(*strides)
    kv = _kv(a, p)
    return lib.nsa_paged_attn(V(p["q"]), kv if cache else None, V(p["table"]), V(p["pos"]), V(p["o"]),
                              V(p["lse"]), a["B"], a["M"], a["H"], a["G"], a["D"], a["ps"], a["cols"],
                              a["left"], a["sinks"], 0.0, a["dtype"], s, V(p["ws"]), ws_bytes, None)


BAD = [
    (dict(B=-1), -2), (dict(M=-1), -2), (dict(G=0), -2), (dict(G=65537, H=65537), -2),
    (dict(D=96), -4), (dict(D=0), -4), (dict(ps=-1), -2), (dict(dtype=2), -11), (dict(dtype=7), -11),
    (dict(B=1 << 16, M=1 << 15), -2), (dict(M=(1 << 30) + 1), -2),
    (dict(pages=0), -2), (dict(pages=-4), -2), (dict(pages=1 << 31), -2), (dict(cols=0), -2),
    (dict(cols=-1), -2), (dict(page=8), -13), (dict(page=0), -13), (dict(page=48), -13),
    (dict(page=2048), -13), (dict(cols=1 << 25, page=64), -2), (dict(bits=8), -11), (dict(bits=0), -11),
    (dict(cstr=(4, 8, 8, 8, 8, 8)), -6), (dict(cstr=(8, 8, -8, 8, 8, 8)), -2),
    (dict(cstr=(8, 8, 8, 8, 8, (1 << 36) + 8)), -2),
]


@pytest.mark.parametrize("over,status", BAD)
def test_bad_sizes_and_types(lib, over, status):
    assert _append(lib, **over) == status
    assert _read(lib, **over) == status
    assert _attn(lib, **over) == status


@pytest.mark.parametrize("over,status", [
    (dict(H=-1), -2), (dict(R=24), -2), (dict(R=144), -2), (dict(rows=-1), -2), (dict(wdtype=0), -11),
    (dict(eps=float("nan")), -2), (dict(eps=float("inf")), -2),
    (dict(eps=-1.0), -2),  # no norm, but weights
    (dict(cstr=(0, 8, 8, 8, 8, 8)), -2), (dict(cstr=(8, 8, 8, 8, 0, 8)), -2)])
def test_append_refuses(lib, over, status):
    assert _append(lib, **over) == status


def test_attention_refuses(lib):
    assert _attn(lib, H=15) == -5
    assert _attn(lib, sinks=-1) == -2
    need = _lib.paged_attn_workspace_bytes(2, 3, 16, 2, 128, 100 * 64)
    assert need > 0
    assert _attn(lib, cols=100, ws_bytes=need - 1) == -9
    assert _attn(lib, {"ws": None}, cols=100) == -9
    assert _attn(lib, {"ws": FAKE + 8}, cols=100) == -6
    assert _attn(lib, strides=[8 * 16 * 128 + 4, 16 * 128, 128]) == -6
    assert _attn(lib, strides=[-8, 16 * 128, 128]) == -2
    assert _attn(lib, strides=[0, 16 * 128, 128]) == -2


@pytest.mark.parametrize("which", ["k", "v", "q", "qo", "kp", "vp", "table", "cos", "sin"])
def test_append_null_and_misaligned(lib, which):
    assert _append(lib, {which: None}) == -1
    assert _append(lib, {which: FAKE + 2}) == -6


@pytest.mark.parametrize("which", ["k", "v", "kp", "vp", "table", "pos"])
def test_read_null_and_misaligned(lib, which):
    assert _read(lib, {which: None}) == -1
    assert _read(lib, {which: FAKE + 2}) == -6


@pytest.mark.parametrize("which", ["q", "kp", "vp", "table", "pos", "o"])
def test_attention_null_and_misaligned(lib, which):
    assert _attn(lib, {which: None}) == -1
    assert _attn(lib, {which: FAKE + 2}) == -6
    assert _attn(lib, {"lse": FAKE + 2}) == -6


@pytest.mark.parametrize("which", ["ks", "vs"])
def test_four_bits_need_scales(lib, which):
    for call in (_append, _read, _attn):
        assert call(lib, {which: None}, bits=4) == -1
        assert call(lib, {which: FAKE + 4}, bits=4) == -6


def test_no_cache(lib):
    for call in (_append, _read, _attn):
        assert call(lib, cache=False) == -1


def test_empty_problem_is_a_no_op(lib):
    none = dict.fromkeys(_ptrs(None))
    for call in (_append, _read, _attn):
        assert call(lib, none, B=0) == 0 and call(lib, none, M=0) == 0


def test_workspace_sizes(lib):
    f = _lib.paged_attn_workspace_bytes
    assert f(1, 1, 64, 8, 128, 512) == 0  # one CTA an item
    assert 0 < f(1, 1, 64, 8, 128, 513) <= 20 << 20
    assert f(64, 1, 64, 8, 128, 2048) == 0 and f(64, 1, 64, 8, 128, 2049) > 0
    assert f(1, 1, 64, 8, 128, 1 << 20, (400, 0), 4) == 0  # what a window leaves to be seen
    assert f(1, 2, 64, 8, 128, 1 << 20, (400, 0), 4) > 0   # (two queries may be far apart)
    assert f(513, 1, 8, 1, 64, 1 << 20) == 0  # items enough
    assert f(0, 1, 8, 1, 64, 1 << 20) == 0
    for bad, status in (((1, 1, 9, 2, 64, 100), -5), ((1, 1, 8, 1, 80, 100), -4),
                        ((-1, 1, 8, 1, 64, 100), -2), ((1, 1, 8, 1, 64, -1), -2)):
        assert lib.nsa_paged_attn_workspace_bytes(*bad, -1, 0) == status
    with pytest.raises(_lib.NsaError):
        f(1, 1, 9, 2, 64, 100)


def test_status_string(lib):
    assert "page_size" in lib.nsa_status_string(-13).decode()


def test_binding_refuses():
    import torch

    from nsa_block_selection_gb300 import KvCache, kv_cache

    k = torch.zeros(4, 16, 2, 64).bfloat16()
    with pytest.raises(ValueError):  # not on a GPU
        KvCache(k, k)
    with pytest.raises(ValueError):
        KvCache(k, k[:2])
    with pytest.raises(TypeError):
        KvCache(k.float(), k.float())
    with pytest.raises(ValueError):
        KvCache(k, k.half())
    with pytest.raises(ValueError):  # one scale
        KvCache(k, k, torch.zeros(4, 2, 16, 2).bfloat16())
    with pytest.raises(ValueError):
        kv_cache(4, 16, 2, 64, bits=8, device="cpu")
    c = torch.zeros(4, 16, 2, 32, dtype=torch.uint8)
    with pytest.raises(TypeError):
        KvCache(c, c, torch.zeros(4, 2, 16, 2), torch.zeros(4, 2, 16, 2))
    with pytest.raises(ValueError):
        KvCache(c, c, *(torch.zeros(4, 16, 2, 2).bfloat16() for _ in range(2)))


# ---- the oracle

def test_quantise_by_hand():
    code, step, low = P.quantise(np.array([[-1.0, 0.0, 0.5, 2.0], [3.0, 3.0, 3.0, 3.0]]))
    assert low[0, 0] == -1 and step[0, 0] == np.float64(0.2001953125)  # 3 / 15 as bf16
    assert code[0].tolist() == [0, 5, 7, 15]
    assert low[1, 0] == 3 and step[1, 0] == 0 and code[1].tolist() == [0] * 4


def test_quantise_is_within_half_a_step():
    x = np.random.default_rng(0).normal(size=(50, 64))
    code, step, low = P.quantise(x)
    # (the two ends are rounded to 8 bits: half a unit of each more)
    slack = step / 2 + 2.0 ** -8 * (np.abs(low) + 15 * step)
    assert (np.abs(low + step * code - x) <= slack).all()
    assert code.min() >= 0 and code.max() <= 15


def test_places():
    assert P.place([7, -1, 3], 0, 16, 8) == (7, 0)
    assert P.place([7, -1, 3], 47, 16, 8) == (3, 15)
    assert P.place([7, -1, 3], 20, 16, 8) is None
    assert P.place([7, -1, 3], 48, 16, 8) is None
    assert P.place([8], 0, 16, 8) is None and P.place([7], -1, 16, 8) is None


def test_attend_is_the_library_attention():
    import torch

    rng = np.random.default_rng(1)
    q, k, v = rng.normal(size=(3, 4, 8)), rng.normal(size=(9, 2, 8)), rng.normal(size=(9, 2, 8))
    present = np.ones(9, bool)
    present[4] = False
    pos, left, sinks = np.array([8, 2, 6]), 3, 2
    o, lse, mag, seen = P.attend(q, k, v, present, pos, left, sinks, 0.3)
    j = np.arange(9)
    mask = np.stack([(j <= p) & ((j >= p - left) | (j < sinks)) & present for p in pos])
    assert (seen == mask.sum(1)).all()
    t = lambda x: torch.from_numpy(x).permute(1, 0, 2)  # noqa: E731
    want = torch.nn.functional.scaled_dot_product_attention(
        t(q), t(np.repeat(k, 2, 1)), t(np.repeat(v, 2, 1)), attn_mask=torch.from_numpy(mask), scale=0.3)
    assert np.abs(want.permute(1, 0, 2).numpy() - o).max() < 1e-12
    assert (mag >= np.abs(o) - 1e-12).all()
    s = np.einsum("mhd,nhd->hmn", q, np.repeat(k, 2, 1)) * 0.3
    assert np.abs(np.log(np.where(mask, np.exp(s), 0).sum(-1)) - lse).max() < 1e-12


def test_attend_without_a_key():
    o, lse, _, seen = P.attend(np.ones((2, 1, 4)), np.ones((3, 1, 4)), np.ones((3, 1, 4)),
                               np.zeros(3, bool), np.array([2, -1]), -1, 0, 1.0)
    assert (o == 0).all() and (lse == -np.inf).all() and (seen == 0).all()
