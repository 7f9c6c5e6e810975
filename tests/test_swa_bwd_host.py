"""Refusals, the workspace size and empty problems of nsa_swa_bwd (no GPU:
arguments are rejected before any CUDA call)."""

import ctypes
import os

import pytest

from nsa_block_selection_gb300 import _lib

FAKE = 4096  # a 16-byte aligned non-null address that is never dereferenced
GOOD = dict(B=2, M=300, N=300, H=16, G=2, D=128, left=64, right=0, dtype=1, gdtype=1)
NAMES = ("q", "k", "v", "o", "lse", "do", "dq", "dk", "dv")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from nsa_block_selection_gb300.build import build

        build()
    return _lib.load()


def _call(lib, ptrs=None, ws=FAKE, ws_bytes=1 << 40, **over):
    a = dict(GOOD, **over)
    p = dict.fromkeys(NAMES, FAKE)
    p.update(ptrs or {})
    return lib.nsa_swa_bwd(*(ctypes.c_void_p(p[n]) for n in NAMES), a["B"], a["M"], a["N"], a["H"],
                           a["G"], a["D"], a["left"], a["right"], 0.0, a["dtype"], a["gdtype"],
                           ctypes.c_void_p(ws), ws_bytes, None)


@pytest.mark.parametrize("over,status", [
    (dict(B=-1), -2), (dict(M=-1), -2), (dict(N=-1), -2), (dict(H=0), -2), (dict(G=0), -2),
    (dict(H=15), -5), (dict(D=96), -4), (dict(D=256), -4), (dict(dtype=2), -11),
    (dict(gdtype=0), -11), (dict(gdtype=3), -11), (dict(M=(1 << 29) + 1), -2),
    (dict(N=(1 << 29) + 1), -2), (dict(H=65538), -2), (dict(B=65537), -2),
    (dict(B=1 << 12, M=1 << 25), -2), (dict(B=1 << 12, N=1 << 25), -2),
])
def test_bad_sizes_and_types(lib, over, status):
    assert _call(lib, **over) == status


@pytest.mark.parametrize("which", NAMES)
def test_null_and_misaligned(lib, which):
    assert _call(lib, {which: None}) == -1
    assert _call(lib, {which: FAKE + 2}) == -6


def test_workspace(lib):
    f = lib.nsa_swa_bwd_workspace_bytes
    stat = 2 * 2 * 16 * 320 * 4
    tile = 2 * 128 * 128 * 4  # fp32 dK and dV of 128 keys
    # 12 key tiles of (batch, KV head), 3 query blocks x 8 heads = 24 steps each:
    # cut into 6 parts of 4
    assert f(2, 300, 300, 16, 2, 128, 64, 0) == stat + 12 * 6 * tile
    # 8 x 64 tiles = 3 rounds of 152 and 56 more, cut in two
    assert f(1, 8192, 8192, 64, 8, 128, 512, 0) == 2 * 64 * 8192 * 4 + 56 * 2 * tile
    # uneven tiles, more than the SMs: whole
    assert f(1, 8192, 8192, 64, 8, 128, -1, 0) == 2 * 64 * 8192 * 4
    # 8 query tiles of 512 steps, cut into 19 parts, one for each SM, beside
    # 256 key tiles of 16 steps: 152 and 104 more, whole
    assert f(1, 128, 32768, 8, 1, 128, -1, -1) == 2 * 8 * 128 * 4 + 8 * 19 * tile // 2
    assert f(1, 0, 300, 16, 2, 128, -1, -1) == 0 and f(1, 300, 0, 16, 2, 128, -1, -1) == 0
    assert f(1, 300, 300, 15, 2, 128, -1, -1) == -5 and f(1, 300, 300, 16, 2, 80, -1, -1) == -4
    need = f(2, 300, 300, 16, 2, 128, 64, 0)
    assert _call(lib, ws_bytes=need - 1) == -9
    assert _call(lib, ws=None) == -9
    assert _call(lib, ws=FAKE + 8) == -6


def test_no_batch_is_a_no_op(lib):
    assert _call(lib, dict.fromkeys(NAMES), ws=None, ws_bytes=0, B=0) == 0
    assert _call(lib, dict.fromkeys(NAMES), ws=None, ws_bytes=0, M=0, N=0) == 0


def test_binding_refuses():
    import torch

    from nsa_block_selection_gb300 import swa_bwd

    q, k = torch.zeros(1, 8, 4, 64).bfloat16(), torch.zeros(1, 8, 2, 64).bfloat16()
    lse = torch.zeros(1, 4, 8)
    with pytest.raises(TypeError):
        swa_bwd(q.float(), k, k, q, lse, q)
    with pytest.raises(TypeError):
        swa_bwd(q, k, k.half(), q, lse, q)
    with pytest.raises(TypeError):
        swa_bwd(q, k, k, q, lse, q, grad_dtype=torch.float16)
    with pytest.raises(ValueError):
        swa_bwd(q, k, k, q, lse[:, :, :7], q)
    with pytest.raises(ValueError):  # not on a GPU
        swa_bwd(q, k, k, q, lse, q)


def test_stream_of_another_device_is_refused():
    import types

    import torch

    from nsa_block_selection_gb300 import swa_bwd

    q, k = torch.zeros(1, 8, 4, 64).bfloat16(), torch.zeros(1, 8, 2, 64).bfloat16()
    other = types.SimpleNamespace(device=torch.device("cuda:7"))
    with pytest.raises(ValueError, match="stream"):
        swa_bwd(q, k, k, q, torch.zeros(1, 4, 8), q, stream=other)
