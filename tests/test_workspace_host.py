"""Workspaces that hold less memory than they have entries are refused (no GPU:
stand-ins for device tensors, which nothing dereferences)."""

import pytest
import torch

from nsa_block_selection_gb300 import _lib


class Device:
    """What the binding asks of a tensor on device 0."""

    def __init__(self, t):
        self.t = t
        self.dtype, self.shape, self.device = t.dtype, t.shape, torch.device("cuda:0")

    def get_device(self):
        return 0

    def data_ptr(self):
        return 4096

    def __getattr__(self, name):
        return getattr(self.t, name)


def _repeated(nbytes):
    """One byte of memory, seen `nbytes` times."""
    return Device(torch.zeros(1, dtype=torch.uint8).expand(nbytes))


def test_swa_bwd():
    q, k = Device(torch.zeros(1, 8, 4, 64).half()), Device(torch.zeros(1, 8, 2, 64).half())
    lse = Device(torch.zeros(1, 4, 8))
    need = _lib.swa_bwd_workspace_bytes(1, 8, 8, 4, 2, 64)
    with pytest.raises(ValueError, match="workspace"):
        _lib.swa_bwd(q, k, k, q, lse, q, dq=q, dk=k, dv=k, workspace=_repeated(need))


def test_norm_rope_bwd():
    q, k = Device(torch.zeros(1, 8, 4, 64).half()), Device(torch.zeros(1, 8, 2, 64).half())
    w = Device(torch.zeros(64))
    need = _lib.norm_rope_bwd_workspace_bytes(1, 8, 64)
    with pytest.raises(ValueError, match="workspace"):
        _lib.qk_norm_rope_bwd(q, k, q, k, dq=q, dk=k, dq_weight=w, dk_weight=w,
                              workspace=_repeated(need))
