"""Refusals and empty problems of the norm-and-rotation entry points (no GPU:
arguments are rejected before any CUDA call), and the angle tables."""

import ctypes

import numpy as np
import pytest

from nsa_block_selection_gb300 import _lib

FAKE = 4096  # a 16-byte aligned non-null address that is never dereferenced
GOOD = dict(B=2, M=100, H=16, G=2, D=128, R=128, rows=100, ps=100, eps=1e-6, inter=0, dtype=1,
            wdtype=2, gdtype=2)


@pytest.fixture(scope="module")
def lib():
    import os

    if not os.path.exists(_lib.LIB_PATH):
        from nsa_block_selection_gb300.build import build

        build()
    return _lib.load()


def _fwd(lib, ptrs=None, strides=None, **over):
    a = dict(GOOD, **over)
    names = ("q", "k", "qo", "ko", "wq", "wk", "cos", "sin", "pos")
    p = dict.fromkeys(names, FAKE)
    p.update(ptrs or {})
    s = None if strides is None else (ctypes.c_int64 * 12)(*strides)
    return lib.nsa_qk_norm_rope(*(ctypes.c_void_p(p[n]) for n in names), a["B"], a["M"], a["H"],
                                a["G"], a["D"], a["R"], a["rows"], a["ps"], a["eps"], a["inter"],
                                a["dtype"], a["wdtype"], s, None)


def _bwd(lib, ptrs=None, strides=None, ws=FAKE, ws_bytes=1 << 30, **over):
    a = dict(GOOD, **over)
    names = ("q", "k", "gq", "gk", "dq", "dk", "dwq", "dwk", "wq", "wk", "cos", "sin", "pos")
    p = dict.fromkeys(names, FAKE)
    p.update(ptrs or {})
    s = None if strides is None else (ctypes.c_int64 * 18)(*strides)
    return lib.nsa_qk_norm_rope_bwd(*(ctypes.c_void_p(p[n]) for n in names), a["B"], a["M"],
                                    a["H"], a["G"], a["D"], a["R"], a["rows"], a["ps"], a["eps"],
                                    a["inter"], a["dtype"], a["wdtype"], a["gdtype"], s,
                                    ctypes.c_void_p(ws), ws_bytes, None)


BAD = [
    (dict(B=-1), -2), (dict(M=-1), -2), (dict(H=0), -2), (dict(G=0), -2), (dict(H=65537), -2),
    (dict(D=96), -4), (dict(D=0), -4), (dict(R=-16), -2), (dict(R=144), -2), (dict(R=24), -2),
    (dict(rows=-1), -2), (dict(rows=(1 << 31) + 1), -2), (dict(ps=-1), -2),
    (dict(eps=-1e-6), -2), (dict(eps=float("nan")), -2), (dict(eps=float("inf")), -2),
    (dict(B=1 << 16, M=1 << 15), -2), (dict(M=(1 << 30) + 1), -2),
    (dict(dtype=2), -11), (dict(dtype=3), -11), (dict(wdtype=0), -11),
]


@pytest.mark.parametrize("over,status", BAD)
def test_bad_sizes_and_types(lib, over, status):
    assert _fwd(lib, **over) == status
    assert _bwd(lib, **over) == status


def test_gradient_type_and_workspace(lib):
    assert _bwd(lib, gdtype=0) == -11
    assert _bwd(lib, ws=None) == -9
    assert _bwd(lib, ws=FAKE + 8) == -6
    need = _lib.norm_rope_bwd_workspace_bytes(2, 100, 128)
    assert _bwd(lib, ws_bytes=need - 1) == -9
    f = lib.nsa_qk_norm_rope_bwd_workspace_bytes
    assert f(2, 100, 128) == 456 * 128 * 4
    assert f(1, 1 << 20, 64) == 456 * 64 * 4
    assert f(1, 100, 80) == -4 and f(-1, 100, 64) == -2 and f(0, 0, 64) == 0


@pytest.mark.parametrize("which", ["q", "k", "qo", "ko", "cos", "sin"])
def test_null_and_misaligned(lib, which):
    assert _fwd(lib, {which: None}) == -1
    assert _fwd(lib, {which: FAKE + 8}) == -6


@pytest.mark.parametrize("which", ["q", "k", "gq", "gk", "dq", "dk", "cos", "sin"])
def test_null_and_misaligned_bwd(lib, which):
    assert _bwd(lib, {which: None}) == -1
    assert _bwd(lib, {which: FAKE + 8}) == -6


def test_small_pointers(lib):
    assert _fwd(lib, {"wq": FAKE + 8}) == -6
    assert _fwd(lib, {"pos": FAKE + 2}) == -6
    assert _bwd(lib, {"wk": FAKE + 8}) == -6
    assert _bwd(lib, {"dwq": FAKE + 2}) == -6


def test_table_shorter_than_the_sequence(lib):
    # token m at position m: the table has to hold every one
    assert _fwd(lib, {"pos": None}, rows=99) == -2
    assert _bwd(lib, {"pos": None}, rows=99) == -2


def test_strides(lib):
    good = [20 * 128 * 100, 20 * 128, 128] * 4
    for n, call, total in ((4, _fwd, 12), (6, _bwd, 18)):
        s = good[:3] * n
        for bad, status in ((4, -6), (-8, -2), ((1 << 40) + 8, -2)):
            for at in (0, 4, total - 1):
                t = list(s)
                t[at] = bad
                assert call(lib, strides=t) == status
        t = list(s)
        t[total - 1] = 0  # all the heads of a written tensor in one place
        assert call(lib, strides=t) == -2


def test_empty_problem_is_a_no_op(lib):
    none = dict.fromkeys(("q", "k", "qo", "ko"))
    assert _fwd(lib, none, B=0) == 0 and _fwd(lib, none, M=0) == 0
    none = dict.fromkeys(("q", "k", "gq", "gk", "dq", "dk", "dwq", "dwk"))
    assert _bwd(lib, none, B=0) == 0 and _bwd(lib, none, M=0) == 0


def test_binding_refuses():
    import torch

    from nsa_block_selection_gb300 import qk_norm_rope, qk_norm_rope_bwd

    q, k = torch.zeros(1, 2, 4, 64).bfloat16(), torch.zeros(1, 2, 1, 64).bfloat16()
    with pytest.raises(TypeError):
        qk_norm_rope(q.float(), k.float())
    with pytest.raises(TypeError):
        qk_norm_rope(q, k.half())
    with pytest.raises(ValueError):
        qk_norm_rope(q, k[:, :1])
    with pytest.raises(ValueError):  # not on a GPU
        qk_norm_rope(q, k)
    with pytest.raises(TypeError):
        qk_norm_rope_bwd(q, k, q.float(), k)


def test_rope_tables():
    from nsa_block_selection_gb300 import rope_tables

    cos, sin = rope_tables(70000, 64, base=500000.0, device="cpu")
    assert cos.shape == sin.shape == (70000, 32)
    i, p = 7, 69999
    ang = p * 500000.0 ** (-2 * i / 64)
    assert abs(cos[p, i].item() - np.cos(ang)) < 2 ** -24
    assert abs(sin[p, i].item() - np.sin(ang)) < 2 ** -24
    with pytest.raises(ValueError):
        rope_tables(10, 7)


def test_stream_of_another_device_is_refused():
    """Before anything is launched or made current."""
    import types

    import torch

    from nsa_block_selection_gb300 import qk_norm_rope, qk_norm_rope_bwd

    q, k = torch.zeros(1, 4, 2, 64).half(), torch.zeros(1, 4, 1, 64).half()
    other = types.SimpleNamespace(device=torch.device("cuda:7"))
    with pytest.raises(ValueError, match="stream"):
        qk_norm_rope(q, k, stream=other)
    with pytest.raises(ValueError, match="stream"):
        qk_norm_rope(q=q, k=k, stream=other)
    with pytest.raises(ValueError, match="stream"):
        qk_norm_rope_bwd(q, k, q, k, stream=other)
