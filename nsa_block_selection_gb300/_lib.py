"""ctypes binding of ``libnsa_sel_attn.so`` (argument marshalling only).

Every step of the selection-attention forward runs in the library's CUDA
kernels; this module only checks tensor dtypes/devices, allocates outputs
with torch and passes raw pointers, sizes and the current CUDA stream. There
is no fallback: if the library is missing, calls raise.
"""

from __future__ import annotations

import ctypes
import os
from array import array
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "lib", "libnsa_sel_attn.so")

NSA_OK = 0
NSA_F16, NSA_BF16, NSA_F32 = 0, 1, 2

EXPORTS = ("nsa_status_string", "nsa_version", "nsa_sel_attn_fwd", "nsa_sel_attn_fwd_ex",
           "nsa_sel_attn_fwd_strided", "nsa_sync_status",
           "nsa_selftest_wait_timeout", "nsa_sel_attn_fwd_host_workspace_bytes",
           "nsa_sel_attn_fwd_host", "nsa_sel_attn_bwd_workspace_bytes", "nsa_sel_attn_bwd",
           "nsa_sel_attn_bwd_noalloc", "nsa_topk_blocks", "nsa_swa_fwd",
           "nsa_sel_attn_fwd_shared_workspace_bytes", "nsa_sel_attn_fwd_shared",
           "nsa_probe_l2_gather", "nsa_probe_l2_gather_bytes", "nsa_probe_gather_rows",
           "nsa_probe_reduce_rows", "nsa_sel_attn_fwd_host_ex", "nsa_sel_attn_bwd_ex",
           "nsa_qk_norm_rope", "nsa_qk_norm_rope_bwd", "nsa_qk_norm_rope_bwd_workspace_bytes",
           "nsa_swa_bwd", "nsa_swa_bwd_workspace_bytes", "nsa_kv_append", "nsa_kv_read",
           "nsa_paged_attn", "nsa_paged_attn_workspace_bytes")

_lib = None


class NsaError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what} failed: {status_string(status)} ({status})")
        self.status = status


def load(path: Optional[str] = None) -> ctypes.CDLL:
    """Load the library (once) and declare the C signatures."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(
            f"{p} is missing: build it with `python -m nsa_block_selection_gb300.build` "
            "(the CUDA library is the only implementation)")
    lib = ctypes.CDLL(p)
    i64, c_int, vp = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
    lib.nsa_status_string.restype = ctypes.c_char_p
    lib.nsa_status_string.argtypes = [c_int]
    lib.nsa_version.restype = c_int
    lib.nsa_version.argtypes = []
    lib.nsa_sel_attn_fwd.restype = c_int
    lib.nsa_sel_attn_fwd.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i64, i64,
                                     c_int, ctypes.c_float, vp]
    lib.nsa_sel_attn_fwd_ex.restype = c_int
    lib.nsa_sel_attn_fwd_ex.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i64,
                                        i64, c_int, ctypes.c_float, c_int, c_int, vp]
    lib.nsa_sel_attn_fwd_strided.restype = c_int
    lib.nsa_sel_attn_fwd_strided.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64,
                                             i64, i64, c_int, ctypes.c_float, c_int, c_int, vp,
                                             vp]
    lib.nsa_sel_attn_fwd_shared_workspace_bytes.restype = i64
    lib.nsa_sel_attn_fwd_shared_workspace_bytes.argtypes = [i64, i64, i64]
    lib.nsa_sel_attn_fwd_shared.restype = c_int
    lib.nsa_sel_attn_fwd_shared.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i64,
                                            i64, c_int, ctypes.c_float, c_int, vp, i64, vp]
    lib.nsa_sync_status.restype = c_int
    lib.nsa_sync_status.argtypes = [vp]
    lib.nsa_selftest_wait_timeout.restype = c_int
    lib.nsa_selftest_wait_timeout.argtypes = [i64, vp]
    lib.nsa_sel_attn_fwd_host_workspace_bytes.restype = i64
    lib.nsa_sel_attn_fwd_host_workspace_bytes.argtypes = [i64, i64, i64, i64, i64, i64, i64,
                                                          c_int, i64]
    lib.nsa_sel_attn_bwd_workspace_bytes.restype = i64
    lib.nsa_sel_attn_bwd_workspace_bytes.argtypes = [i64, i64, i64, i64, i64, i64, i64, c_int]
    lib.nsa_sel_attn_bwd.restype = c_int
    lib.nsa_sel_attn_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64,
                                     i64, i64, i64, c_int, ctypes.c_float, vp, i64, vp]
    lib.nsa_sel_attn_bwd_ex.restype = c_int
    lib.nsa_sel_attn_bwd_ex.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64,
                                        i64, i64, i64, i64, c_int, ctypes.c_float, c_int, vp, i64,
                                        vp]
    lib.nsa_sel_attn_bwd_noalloc.restype = c_int
    lib.nsa_sel_attn_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i64,
                                             i64, i64, i64, i64, i64, c_int, ctypes.c_float, vp]
    lib.nsa_swa_fwd.restype = c_int
    lib.nsa_swa_fwd.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i64, i64, i64,
                                ctypes.c_float, c_int, vp]
    lib.nsa_topk_blocks.restype = c_int
    lib.nsa_topk_blocks.argtypes = [vp, vp, i64, i64, i64, i64, i64, c_int, c_int, c_int, vp]
    lib.nsa_sel_attn_fwd_host_ex.restype = c_int
    lib.nsa_sel_attn_fwd_host_ex.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64,
                                             i64, i64, c_int, ctypes.c_float, c_int, c_int, vp,
                                             i64, i64, vp]
    lib.nsa_sel_attn_fwd_host.restype = c_int
    lib.nsa_sel_attn_fwd_host.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i64,
                                          i64, c_int, ctypes.c_float, vp, i64, i64, vp]
    lib.nsa_probe_l2_gather.restype = c_int
    lib.nsa_probe_l2_gather.argtypes = [vp, vp, i64, i64, i64, i64, c_int, i64, c_int, c_int,
                                        i64, c_int, ctypes.c_uint32, vp, vp]
    lib.nsa_probe_l2_gather_bytes.restype = i64
    lib.nsa_probe_l2_gather_bytes.argtypes = [i64, i64, c_int, i64, c_int]
    lib.nsa_probe_reduce_rows.restype = c_int
    lib.nsa_probe_reduce_rows.argtypes = [vp, i64, i64, i64, c_int, i64, ctypes.c_uint32, vp]
    lib.nsa_probe_gather_rows.restype = c_int
    lib.nsa_probe_gather_rows.argtypes = [vp, vp, vp, i64, i64, i64, i64, i64, i64, c_int, i64,
                                          c_int, c_int, i64, vp]
    f32 = ctypes.c_float
    lib.nsa_swa_bwd_workspace_bytes.restype = i64
    lib.nsa_swa_bwd_workspace_bytes.argtypes = [i64] * 8
    lib.nsa_swa_bwd.restype = c_int
    lib.nsa_swa_bwd.argtypes = [vp] * 9 + [i64] * 8 + [f32, c_int, c_int, vp, i64, vp]
    lib.nsa_qk_norm_rope.restype = c_int
    lib.nsa_qk_norm_rope.argtypes = [vp] * 9 + [i64] * 8 + [f32, c_int, c_int, c_int, vp, vp]
    lib.nsa_qk_norm_rope_bwd_workspace_bytes.restype = i64
    lib.nsa_qk_norm_rope_bwd_workspace_bytes.argtypes = [i64, i64, i64]
    lib.nsa_qk_norm_rope_bwd.restype = c_int
    lib.nsa_qk_norm_rope_bwd.argtypes = [vp] * 13 + [i64] * 8 + [f32, c_int, c_int, c_int, c_int,
                                                                 vp, vp, i64, vp]
    lib.nsa_kv_append.restype = c_int
    lib.nsa_kv_append.argtypes = [vp] * 11 + [i64] * 9 + [f32, c_int, c_int, c_int, vp, vp]
    lib.nsa_kv_read.restype = c_int
    lib.nsa_kv_read.argtypes = [vp] * 5 + [i64] * 6 + [c_int, vp]
    lib.nsa_paged_attn_workspace_bytes.restype = i64
    lib.nsa_paged_attn_workspace_bytes.argtypes = [i64] * 8
    lib.nsa_paged_attn.restype = c_int
    lib.nsa_paged_attn.argtypes = [vp] * 6 + [i64] * 9 + [f32, c_int, vp, vp, i64, vp]
    if path is None:
        _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().nsa_status_string(int(status)).decode()


def _ptr(t) -> Optional[int]:
    return t.data_ptr() if t is not None and t.numel() > 0 else None


def _dtype_code(dt) -> int:
    import torch

    return {torch.float16: NSA_F16, torch.bfloat16: NSA_BF16, torch.float32: NSA_F32}[dt]


def sel_attn_fwd(q, k, v, block_indices, block_size: int, scale: Optional[float] = None,
                 out=None, lse=None, stream=None, out_dtype=None):
    """NSA selection-attention forward on the GPU.

    q: fp16 or bf16 [B, M, H, D]; k, v: [B, N, G, D] of q's dtype;
    block_indices: int32 [B, M, G, T] (-1 = padding), contiguous; all on one
    CUDA device. q, k, v (and a preallocated ``out``) may be strided views
    (for example slices of one fused projection) whose last dimension is
    contiguous and whose strides are multiples of 8 elements. Returns
    (O [B, M, H, D], LSE fp32 [B, H, M]). O is fp32 unless ``out_dtype`` (or
    a preallocated ``out``) is q's dtype. ``stream`` defaults to torch's
    current stream.
    """
    import torch

    lib = load()
    B, M, N, H, G, D, T = _check_common(q, k, v, block_indices, device_expected=True,
                                        qkv_dtypes=(torch.float16, torch.bfloat16),
                                        strided=True)
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.float32
    if out_dtype not in (torch.float32, q.dtype):
        raise TypeError(f"O must be fp32 or {q.dtype}, got {out_dtype}")
    if out is None:
        out = torch.empty((B, M, H, D), dtype=out_dtype, device=q.device)
    if lse is None:
        lse = torch.empty((B, H, M), dtype=torch.float32, device=q.device)
    if out.dtype != out_dtype or tuple(out.shape) != (B, M, H, D) or out.stride(-1) != 1:
        raise ValueError(f"out must be {out_dtype} [B, M, H, D] with a contiguous last dim")
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, M) or not lse.is_contiguous():
        raise ValueError("lse must be contiguous fp32 [B, H, M]")
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    sc = float(scale) if scale is not None else 0.0  # the ABI: <= 0 selects 1/sqrt(D)
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(block_indices), _ptr(out), _ptr(lse), B, M, N, H,
            G, D, T, int(block_size), sc)
    if not all(t.is_contiguous() or t.numel() == 0 for t in (q, k, v, out)):
        strides = (ctypes.c_int64 * 12)(*(list(q.stride()[:3]) + list(k.stride()[:3]) +
                                          list(v.stride()[:3]) + list(out.stride()[:3])))
        st = lib.nsa_sel_attn_fwd_strided(*args, _dtype_code(q.dtype), _dtype_code(out.dtype),
                                          strides, ctypes.c_void_p(stream.cuda_stream))
        what = "nsa_sel_attn_fwd_strided"
    elif q.dtype == torch.float16 and out.dtype == torch.float32:
        st = lib.nsa_sel_attn_fwd(*args, ctypes.c_void_p(stream.cuda_stream))
        what = "nsa_sel_attn_fwd"
    else:
        st = lib.nsa_sel_attn_fwd_ex(*args, _dtype_code(q.dtype), _dtype_code(out.dtype),
                                     ctypes.c_void_p(stream.cuda_stream))
        what = "nsa_sel_attn_fwd_ex"
    if st != NSA_OK:
        raise NsaError(st, what)
    return out, lse


def shared_workspace_bytes(B, M, G) -> int:
    n = load().nsa_sel_attn_fwd_shared_workspace_bytes(B, M, G)
    if n < 0:
        raise NsaError(int(n), "nsa_sel_attn_fwd_shared_workspace_bytes")
    return int(n)


def sel_attn_fwd_shared(q, k, v, block_indices, block_size: int, scale: Optional[float] = None,
                        out=None, lse=None, workspace=None, stream=None):
    """The two-pass forward (nsa_sel_attn_fwd_shared): blocks common to a tile
    of 16 consecutive queries are gathered once per tile. Contiguous fp16 or
    bf16 q, k, v; O fp32. ``workspace``: a CUDA uint8 tensor of at least
    shared_workspace_bytes(B, M, G) bytes (allocated when None). Returns
    (O, LSE); the per-tile records stay in ``workspace``.
    """
    import torch

    lib = load()
    B, M, N, H, G, D, T = _check_common(q, k, v, block_indices, device_expected=True,
                                        qkv_dtypes=(torch.float16, torch.bfloat16))
    if out is None:
        out = torch.empty((B, M, H, D), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((B, H, M), dtype=torch.float32, device=q.device)
    if out.dtype != torch.float32 or tuple(out.shape) != (B, M, H, D) or not out.is_contiguous():
        raise ValueError("out must be contiguous fp32 [B, M, H, D]")
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, M) or not lse.is_contiguous():
        raise ValueError("lse must be contiguous fp32 [B, H, M]")
    if workspace is None:
        workspace = torch.empty(max(shared_workspace_bytes(B, M, G), 1), dtype=torch.uint8,
                                device=q.device)
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    sc = float(scale) if scale is not None else 0.0  # the ABI: <= 0 selects 1/sqrt(D)
    st = lib.nsa_sel_attn_fwd_shared(_ptr(q), _ptr(k), _ptr(v), _ptr(block_indices), _ptr(out),
                                     _ptr(lse), B, M, N, H, G, D, T, int(block_size), sc,
                                     _dtype_code(q.dtype), _ptr(workspace), workspace.numel(),
                                     ctypes.c_void_p(stream.cuda_stream))
    if st != NSA_OK:
        raise NsaError(st, "nsa_sel_attn_fwd_shared")
    return out, lse


def _check_common(q, k, v, block_indices, device_expected: bool, qkv_dtypes=None,
                  strided: bool = False):
    import torch

    qkv_dtypes = qkv_dtypes or (torch.float16,)
    if q.dtype not in qkv_dtypes:
        raise TypeError(f"q must be one of {qkv_dtypes}, got {q.dtype}")

    B, M, H, D = q.shape
    Bk, N, G, Dk = k.shape
    T = block_indices.shape[-1]
    if (Bk, Dk) != (B, D) or tuple(v.shape) != tuple(k.shape) or \
            tuple(block_indices.shape) != (B, M, G, T):
        raise ValueError("shape mismatch: q [B,M,H,D], k/v [B,N,G,D], "
                         "block_indices [B,M,G,T]")
    named = (("q", q, q.dtype), ("k", k, q.dtype), ("v", v, q.dtype),
             ("block_indices", block_indices, torch.int32))
    for name, t, dt in named:
        if t.dtype != dt:
            raise TypeError(f"{name} must be {dt}, got {t.dtype}")
    for name, t, _ in named:
        if t.is_cuda != device_expected:
            raise ValueError(f"{name} must be a {'CUDA' if device_expected else 'CPU'} tensor")
        if strided and name != "block_indices":
            if t.numel() > 0 and t.stride(-1) != 1:
                raise ValueError(f"{name} must have a contiguous last dimension")
        elif not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    return B, M, N, H, G, D, T


def host_workspace_bytes(B, M, N, H, G, D, T, block_size, chunk_m=0) -> int:
    n = load().nsa_sel_attn_fwd_host_workspace_bytes(B, M, N, H, G, D, T, int(block_size),
                                                     int(chunk_m))
    if n < 0:
        raise NsaError(int(n), "nsa_sel_attn_fwd_host_workspace_bytes")
    return int(n)


def sel_attn_fwd_host(q, k, v, block_indices, block_size: int, scale: Optional[float] = None,
                      out=None, lse=None, chunk_m: int = 0, workspace=None, device=None,
                      stream=None, sync: bool = True, out_dtype=None):
    """Forward with host (CPU) tensors in and out, through the library's
    pipelined host entry point (pin the tensors for overlapped copies).

    q, k, v fp16 or bf16. Returns (O, LSE) as CPU tensors: O fp32 unless
    ``out_dtype`` (or a preallocated ``out``) is q's dtype, LSE fp32.
    ``workspace`` is a CUDA uint8 tensor of at least
    :func:`host_workspace_bytes`; one is allocated when omitted. With
    ``sync=False`` the call returns once everything is enqueued on ``stream``.
    """
    import torch

    lib = load()
    B, M, N, H, G, D, T = _check_common(q, k, v, block_indices, device_expected=False,
                                        qkv_dtypes=(torch.float16, torch.bfloat16))
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.float32
    if out_dtype not in (torch.float32, q.dtype):
        raise TypeError(f"O must be fp32 or {q.dtype}, got {out_dtype}")
    device = torch.device(device) if device is not None else torch.device("cuda",
                                                                        torch.cuda.current_device())
    need = host_workspace_bytes(B, M, N, H, G, D, T, block_size, chunk_m)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=device)
    if out is None:
        out = torch.empty((B, M, H, D), dtype=out_dtype, pin_memory=True)
    if lse is None:
        lse = torch.empty((B, H, M), dtype=torch.float32, pin_memory=True)
    if out.is_cuda or lse.is_cuda or out.dtype != out_dtype or lse.dtype != torch.float32:
        raise ValueError(f"out must be a {out_dtype} CPU tensor and lse an fp32 one")
    if tuple(out.shape) != (B, M, H, D) or tuple(lse.shape) != (B, H, M):
        raise ValueError("out must be [B, M, H, D] and lse [B, H, M]")
    if stream is None:
        stream = torch.cuda.current_stream(device)
    sc = float(scale) if scale is not None else 0.0  # the ABI: <= 0 selects 1/sqrt(D)
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(block_indices), _ptr(out), _ptr(lse), B, M, N, H,
            G, D, T, int(block_size), sc)
    tail = (workspace.data_ptr(), workspace.numel(), int(chunk_m),
            ctypes.c_void_p(stream.cuda_stream))
    if q.dtype == torch.float16 and out.dtype == torch.float32:
        st = lib.nsa_sel_attn_fwd_host(*args, *tail)
        what = "nsa_sel_attn_fwd_host"
    else:
        st = lib.nsa_sel_attn_fwd_host_ex(*args, _dtype_code(q.dtype), _dtype_code(out.dtype),
                                          *tail)
        what = "nsa_sel_attn_fwd_host_ex"
    if st != NSA_OK:
        raise NsaError(st, what)
    if sync:
        stream.synchronize()
    return out, lse


def bwd_workspace_bytes(B, M, N, H, G, D, T, block_size) -> int:
    n = load().nsa_sel_attn_bwd_workspace_bytes(B, M, N, H, G, D, T, int(block_size))
    if n < 0:
        raise NsaError(int(n), "nsa_sel_attn_bwd_workspace_bytes")
    return int(n)


def sel_attn_bwd(q, k, v, block_indices, o, lse, do, block_size: int,
                 scale: Optional[float] = None, dq=None, dk=None, dv=None, workspace=None,
                 stream=None):
    """Gradients of :func:`sel_attn_fwd`: returns (dQ, dK, dV) fp32 CUDA tensors.

    q, k, v fp16 or bf16 (as passed to the forward). ``o`` and ``lse`` are
    the forward's fp32 outputs, ``do`` the fp32 upstream gradient
    [B, M, H, D]. ``workspace`` (CUDA uint8) is allocated when omitted.
    """
    import torch

    lib = load()
    B, M, N, H, G, D, T = _check_common(q, k, v, block_indices, device_expected=True,
                                        qkv_dtypes=(torch.float16, torch.bfloat16))
    for name, t, shape in (("o", o, (B, M, H, D)), ("lse", lse, (B, H, M)),
                           ("do", do, (B, M, H, D))):
        if t.dtype != torch.float32 or tuple(t.shape) != shape or not t.is_contiguous() \
                or not t.is_cuda:
            raise ValueError(f"{name} must be a contiguous fp32 CUDA tensor of shape {shape}")
    dev = q.device
    dq = torch.empty((B, M, H, D), dtype=torch.float32, device=dev) if dq is None else dq
    dk = torch.empty((B, N, G, D), dtype=torch.float32, device=dev) if dk is None else dk
    dv = torch.empty((B, N, G, D), dtype=torch.float32, device=dev) if dv is None else dv
    need = bwd_workspace_bytes(B, M, N, H, G, D, T, block_size)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    sc = float(scale) if scale is not None else 0.0  # the ABI: <= 0 selects 1/sqrt(D)
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(block_indices), _ptr(o), _ptr(lse), _ptr(do),
            _ptr(dq), _ptr(dk), _ptr(dv), B, M, N, H, G, D, T, int(block_size), sc)
    tail = (workspace.data_ptr(), workspace.numel(), ctypes.c_void_p(stream.cuda_stream))
    if q.dtype == torch.float16:
        st = lib.nsa_sel_attn_bwd(*args, *tail)
        what = "nsa_sel_attn_bwd"
    else:
        st = lib.nsa_sel_attn_bwd_ex(*args, _dtype_code(q.dtype), *tail)
        what = "nsa_sel_attn_bwd_ex"
    if st != NSA_OK:
        raise NsaError(st, what)
    return dq, dk, dv


def sync_status(stream=None) -> int:
    """Wait for ``stream`` (default: torch's current stream) and return the
    library's device status (NSA_OK, or -8 after a timed-out device wait)."""
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return load().nsa_sync_status(ctypes.c_void_p(stream.cuda_stream))


def selftest_wait_timeout(limit_ns: int, stream=None) -> int:
    """Launch the self-test kernel whose wait can only time out."""
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return load().nsa_selftest_wait_timeout(int(limit_ns), ctypes.c_void_p(stream.cuda_stream))


def topk_blocks(scores, N: int, block_size: int, T: int, n_init: int = 0, n_local: int = 0,
                out=None, stream=None):
    """Top-k block selection on the GPU (nsa_topk_blocks).

    scores: fp32 [B, M, G, ceil(N/block_size)], contiguous on a CUDA device.
    Returns block_indices int32 [B, M, G, T] (ascending, -1 padded): per
    (b, m, g) the first n_init and last n_local causal blocks and the
    highest-scoring others.
    """
    import torch

    lib = load()
    if scores.dtype != torch.float32 or not scores.is_cuda or not scores.is_contiguous():
        raise TypeError("scores must be a contiguous fp32 CUDA tensor")
    B, M, G, S = scores.shape
    if S != -(-int(N) // int(block_size)):
        raise ValueError("scores must have ceil(N/block_size) entries per row")
    if out is None:
        out = torch.empty((B, M, G, T), dtype=torch.int32, device=scores.device)
    if out.dtype != torch.int32 or tuple(out.shape) != (B, M, G, T) or not out.is_contiguous():
        raise ValueError("out must be contiguous int32 [B, M, G, T]")
    if stream is None:
        stream = torch.cuda.current_stream(scores.device)
    st = lib.nsa_topk_blocks(_ptr(scores), _ptr(out), B, M, int(N), G, int(T), int(block_size),
                             int(n_init), int(n_local), ctypes.c_void_p(stream.cuda_stream))
    if st != NSA_OK:
        raise NsaError(st, "nsa_topk_blocks")
    return out


def swa_fwd(q, k, v, window=(-1, -1), scale: Optional[float] = None, out=None, lse=None,
            return_lse: bool = True, stream=None):
    """GQA sliding-window attention forward on the GPU (nsa_swa_fwd).

    q: bf16 or fp16 [B, M, H, D]; k, v: [B, N, H_kv, D] of q's dtype, all
    contiguous on one CUDA device. ``window`` = (left, right): query i sees
    keys [i - left, i + right]; a negative side is unbounded. Returns
    (O [B, M, H, D] in q's dtype, LSE fp32 [B, H, M] or None). ``stream`` is
    where the kernel runs (default: torch's current stream); outputs that the
    call allocates come from the current stream's memory all the same.
    """
    import torch

    lib = load()
    if q.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError(f"q must be fp16 or bf16, got {q.dtype}")
    for name, t in (("k", k), ("v", v)):
        if t.dtype != q.dtype:
            raise TypeError(f"{name} must be {q.dtype}, got {t.dtype}")
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    B, M, H, D = q.shape
    Bk, N, Hkv, Dk = k.shape
    if (Bk, Dk) != (B, D) or tuple(v.shape) != tuple(k.shape):
        raise ValueError("shape mismatch: q [B,M,H,D], k/v [B,N,H_kv,D]")
    if out is None:
        out = torch.empty((B, M, H, D), dtype=q.dtype, device=q.device)
    if out.dtype != q.dtype or tuple(out.shape) != (B, M, H, D) or not out.is_contiguous():
        raise ValueError(f"out must be contiguous {q.dtype} [B, M, H, D]")
    if lse is None and return_lse:
        lse = torch.empty((B, H, M), dtype=torch.float32, device=q.device)
    if lse is not None and (lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, M)
                            or not lse.is_contiguous()):
        raise ValueError("lse must be contiguous fp32 [B, H, M]")
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    left, right = (int(window[0]), int(window[1])) if window is not None else (-1, -1)
    sc = float(scale) if scale is not None else 0.0  # the ABI: <= 0 selects 1/sqrt(D)
    st = lib.nsa_swa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, M, N, H, Hkv, D,
                         left, right, sc, _dtype_code(q.dtype),
                         ctypes.c_void_p(stream.cuda_stream))
    if st != NSA_OK:
        raise NsaError(st, "nsa_swa_fwd")
    return out, lse


# The calls below may be a single token's work, beside which every property
# read and every import statement counts: torch is looked up once, each
# property is read once, and names are given only where a check failed. _bound
# is the library once torch is there too (load() itself needs no torch).
_bound = None
_torch = None
_F16_KINDS = ()
_DTYPE_CODES = {}


def _bind():
    global _bound, _torch, _F16_KINDS
    import torch

    lib = load()
    _torch = torch
    _F16_KINDS = (torch.float16, torch.bfloat16)
    _DTYPE_CODES.update({torch.float16: NSA_F16, torch.bfloat16: NSA_BF16, torch.float32: NSA_F32})
    _bound = lib
    return lib


def _launch(dev, fn, *args):
    """fn(*args, cudaStream_t) on device ``dev`` and its current stream."""
    c = _torch._C
    if c._cuda_getDevice() == dev:
        return fn(*args, c._cuda_getCurrentRawStream(dev))
    with _torch.cuda.device(dev):
        return fn(*args, c._cuda_getCurrentRawStream(dev))


def _on_stream(stream, call, q, *args):
    """call(q, *args) with ``stream`` current: what the call allocates (a
    workspace that it drops on return among it) then comes from that stream's
    memory, and waits for that stream's work."""
    if stream.device != q.device:
        raise ValueError(f"stream must be one of q's device ({q.device}), got {stream.device}")
    with _torch.cuda.stream(stream):
        return call(q, *args)


def swa_bwd_workspace_bytes(B, M, N, H, H_kv, D, window=(-1, -1)) -> int:
    n = load().nsa_swa_bwd_workspace_bytes(B, M, N, H, H_kv, D, int(window[0]), int(window[1]))
    if n < 0:
        raise NsaError(int(n), "nsa_swa_bwd_workspace_bytes")
    return int(n)


def swa_bwd(q, k, v, o, lse, do, window=(-1, -1), scale: Optional[float] = None, dq=None, dk=None,
            dv=None, grad_dtype=None, workspace=None, *, stream=None):
    """Gradients of :func:`swa_fwd` (nsa_swa_bwd): returns (dQ, dK, dV).

    q, k, v, ``window`` and ``scale`` as passed to the forward, ``o`` and
    ``lse`` what it returned, ``do`` the upstream gradient of o (q's dtype,
    [B, M, H, D]); all contiguous on one CUDA device. The gradients are of
    q's dtype, or fp32 with ``grad_dtype=torch.float32`` (or preallocated
    ones). ``workspace`` (CUDA uint8, swa_bwd_workspace_bytes) is allocated
    when omitted; calls that may overlap need one each. Runs on torch's current
    stream, or on ``stream`` (a keyword; what it allocates is then allocated
    on it too).
    """
    lib = _bound or _bind()
    if stream is not None:
        return _on_stream(stream, swa_bwd, q, k, v, o, lse, do, window, scale, dq, dk, dv,
                          grad_dtype, workspace)
    dt, qs, ks = q.dtype, q.shape, k.shape
    if dt not in _F16_KINDS:
        raise TypeError(f"q must be fp16 or bf16, got {dt}")
    if len(qs) != 4 or len(ks) != 4 or qs[0] != ks[0] or qs[3] != ks[3]:
        raise ValueError("shape mismatch: q [B,M,H,D], k/v [B,N,H_kv,D]")
    B, M, H, D = qs
    N, Hkv = ks[1], ks[2]
    if grad_dtype is None:
        grad_dtype = next((t.dtype for t in (dq, dk, dv) if t is not None), dt)
    if grad_dtype is not _torch.float32 and grad_dtype is not dt:
        raise TypeError(f"gradients must be fp32 or {dt}, got {grad_dtype}")
    like = {} if grad_dtype is dt else {"dtype": grad_dtype}
    if dq is None:
        dq = _torch.empty_like(q, **like)
    if dk is None:
        dk = _torch.empty_like(k, **like)
    if dv is None:
        dv = _torch.empty_like(k, **like)
    named = (("q", q, dt, qs), ("k", k, dt, ks), ("v", v, dt, ks), ("o", o, dt, qs),
             ("lse", lse, _torch.float32, (B, H, M)), ("do", do, dt, qs),
             ("dq", dq, grad_dtype, qs), ("dk", dk, grad_dtype, ks), ("dv", dv, grad_dtype, ks))
    for name, t, want, shape in named:
        if t.dtype is not want:
            raise TypeError(f"{name} must be {want}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must have the shape {tuple(shape)}")
    dev = q.get_device()
    for name, t, _, _ in named:
        if t.get_device() != dev or dev < 0 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous tensor on q's CUDA device")
    left, right = (int(window[0]), int(window[1])) if window is not None else (-1, -1)
    if workspace is None:
        nbytes = lib.nsa_swa_bwd_workspace_bytes(B, M, N, H, Hkv, D, left, right)
        if nbytes < 0:
            raise NsaError(nbytes, "nsa_swa_bwd_workspace_bytes")
        workspace = _torch.empty(nbytes, dtype=_torch.uint8, device=q.device)
    else:
        nbytes = workspace.numel() * workspace.element_size()
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on q's CUDA device")
    # scale: the ABI takes <= 0 for 1/sqrt(D)
    st = _launch(dev, lib.nsa_swa_bwd, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                 o.data_ptr(), lse.data_ptr(), do.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                 dv.data_ptr(), B, M, N, H, Hkv, D, left, right, 0.0 if scale is None else scale,
                 _DTYPE_CODES[dt], _DTYPE_CODES[grad_dtype], workspace.data_ptr(), nbytes)
    if st != NSA_OK:
        raise NsaError(st, "nsa_swa_bwd")
    return dq, dk, dv


def rope_tables(rows: int, rot_dim: int, base: float = 10000.0, device="cuda"):
    """Cosine and sine tables for :func:`qk_norm_rope`: fp32 [rows, rot_dim/2]
    each, the angle of pair i at position p being p * base^(-2i / rot_dim),
    formed in fp64 (an fp32 angle of a far position is off by whole turns'
    fractions). A program builds them once; any other tables of that shape
    (scaled or interpolated positions) serve as well."""
    import torch

    if rows < 0 or rot_dim <= 0 or rot_dim % 2:
        raise ValueError("rows must be >= 0 and rot_dim a positive even number")
    half = rot_dim // 2
    freq = float(base) ** (-torch.arange(half, dtype=torch.float64, device=device) / half)
    ang = torch.arange(rows, dtype=torch.float64, device=device)[:, None] * freq
    return ang.cos().float(), ang.sin().float()


def _at(t):
    return None if t is None else t.data_ptr()


def _dense_like(t):
    """An uninitialised contiguous tensor of t's shape and type."""
    e = _torch.empty_like(t)
    return e if e.is_contiguous() else \
        _torch.empty_like(t, memory_format=_torch.contiguous_format)


def _refuse_tensor(name, t, dtypes, shape, dev):
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {dtypes}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}")
    raise ValueError(f"{name} must be on q's CUDA device, with a contiguous last dimension")


def _check_rope(named, q_weight, k_weight, cos, sin, positions):
    """Checks shared by the norm-and-rotation calls; ``named``: (name, tensor,
    allowed dtypes), of q's and k's shapes in turn. Returns the sizes and codes
    that the calls pass on, and the element strides (None: all contiguous)."""
    q, k = named[0][1], named[1][1]
    dt, qs, ks = q.dtype, q.shape, k.shape
    if dt not in _F16_KINDS:
        raise TypeError(f"q must be fp16 or bf16, got {dt}")
    if len(qs) != 4 or len(ks) != 4 or qs[0] != ks[0] or qs[1] != ks[1] or qs[3] != ks[3]:
        raise ValueError("shape mismatch: q [B,M,H,D], k [B,M,G,D]")
    B, M, H, D = qs
    G = ks[2]
    dev = q.get_device()
    plain = True
    for i, (name, t, dtypes) in enumerate(named):
        if t.dtype not in dtypes or t.shape != (ks if i & 1 else qs):
            _refuse_tensor(name, t, dtypes, ks if i & 1 else qs, dev)
    for i, (name, t, dtypes) in enumerate(named):
        c = t.is_contiguous()
        plain = plain and c
        if t.get_device() != dev or dev < 0 or not (c or t.stride(3) == 1):
            _refuse_tensor(name, t, dtypes, ks if i & 1 else qs, dev)
    strides = None
    if not plain:  # (the stride of a dimension of one is never used)
        strides = array("q")
        for i, (_, t, _) in enumerate(named):
            b, m, h, _ = t.stride()
            strides.extend((b if B > 1 else 0, m if M > 1 else 0,
                            h if (G if i & 1 else H) > 1 else 0))
    wdt = None
    for w in (q_weight, k_weight):
        if w is None:
            continue
        if (w.dtype is not _torch.float32 and w.dtype is not dt) or \
                (wdt is not None and w.dtype is not wdt):
            raise TypeError(f"the weights must be fp32 or {dt}, both alike")
        wdt = w.dtype
        if w.shape != (D,) or not w.is_contiguous() or w.get_device() != dev:
            raise ValueError("a weight must be a contiguous [D] tensor on q's device")
    R = rows = 0
    if cos is not None and sin is not None:
        cs = cos.shape
        if cos.dtype is not _torch.float32 or sin.dtype is not _torch.float32:
            raise TypeError("cos and sin must be fp32")
        if len(cs) != 2 or cs != sin.shape or not cos.is_contiguous() or \
                not sin.is_contiguous() or cos.get_device() != dev or sin.get_device() != dev:
            raise ValueError("cos and sin must be contiguous [rows, R/2] tensors on q's device")
        rows, R = cs[0], 2 * cs[1]
    elif cos is not None or sin is not None:
        raise ValueError("pass both tables or neither")
    pstride = 0
    if positions is not None:
        if positions.dtype is not _torch.int32:
            raise TypeError(f"positions must be int32, got {positions.dtype}")
        ps = positions.shape
        if ps == (B, M):
            pstride = M
        elif ps != (M,):
            raise ValueError("positions must be [M] or [B, M]")
        if not positions.is_contiguous() or positions.get_device() != dev:
            raise ValueError("positions must be a contiguous tensor on q's device")
    return dev, (B, M, H, G, D, R, rows, pstride), _DTYPE_CODES[dt], \
        NSA_F32 if wdt is None else _DTYPE_CODES[wdt], strides


def qk_norm_rope(q, k, q_weight=None, k_weight=None, cos=None, sin=None, positions=None,
                 eps: float = 1e-6, interleaved: bool = False, q_out=None, k_out=None, *,
                 stream=None):
    """RMS norm of every query and key head and the position rotation, in one
    pass (nsa_qk_norm_rope).

    q: fp16 or bf16 [B, M, H, D], k: [B, M, G, D] of q's dtype, D 64 or 128;
    both (and preallocated outputs) may be strided views, such as slices of
    one projection, with a contiguous last dimension and strides that are
    multiples of 8. ``q_weight``, ``k_weight``: [D], fp32 or q's dtype, or None (ones).
    ``cos``, ``sin``: fp32 [rows, R/2] (:func:`rope_tables`); R/2 pairs per
    head are rotated, entries (i, i + R/2), or (2i, 2i + 1) with
    ``interleaved``; None: no rotation. ``positions``: int32 [B, M] or [M]
    table rows of the tokens (None: 0 .. M - 1); a position outside the table
    marks padding, whose output rows are zero. The outputs may be the inputs.
    Runs on torch's current stream, or on ``stream`` (a keyword; the outputs
    are then allocated on it too). Returns (q_out, k_out).
    """
    lib = _bound or _bind()
    if stream is not None:
        return _on_stream(stream, qk_norm_rope, q, k, q_weight, k_weight, cos, sin, positions, eps,
                          interleaved, q_out, k_out)
    if q_out is None:
        q_out = _dense_like(q)
    if k_out is None:
        k_out = _dense_like(k)
    own = (q.dtype,)
    dev, sizes, code, wcode, strides = _check_rope(
        (("q", q, own), ("k", k, own), ("q_out", q_out, own), ("k_out", k_out, own)), q_weight,
        k_weight, cos, sin, positions)
    st = _launch(dev, lib.nsa_qk_norm_rope, q.data_ptr(), k.data_ptr(), q_out.data_ptr(),
                 k_out.data_ptr(), _at(q_weight), _at(k_weight), _at(cos), _at(sin),
                 _at(positions), *sizes, eps, 1 if interleaved else 0, code, wcode,
                 None if strides is None else strides.buffer_info()[0])
    if st != NSA_OK:
        raise NsaError(st, "nsa_qk_norm_rope")
    return q_out, k_out


def norm_rope_bwd_workspace_bytes(B, M, D) -> int:
    n = (_lib or load()).nsa_qk_norm_rope_bwd_workspace_bytes(B, M, D)
    if n < 0:
        raise NsaError(int(n), "nsa_qk_norm_rope_bwd_workspace_bytes")
    return n


def qk_norm_rope_bwd(q, k, dq_out, dk_out, q_weight=None, k_weight=None, cos=None, sin=None,
                     positions=None, eps: float = 1e-6, interleaved: bool = False, dq=None,
                     dk=None, dq_weight=None, dk_weight=None, weight_grads: bool = True,
                     workspace=None, *, stream=None):
    """Gradients of :func:`qk_norm_rope` (nsa_qk_norm_rope_bwd).

    q, k and the arguments after them are the forward's; ``dq_out``,
    ``dk_out`` the gradients of its outputs, fp32 (as :func:`sel_attn_bwd`
    returns them) or q's dtype, both alike; strided views are taken as in
    the forward. Returns (dq, dk, dq_weight, dk_weight): dq, dk of q's dtype,
    the weights' gradients fp32 [D] (None with ``weight_grads=False``).
    ``workspace`` (CUDA uint8, norm_rope_bwd_workspace_bytes) is allocated
    when omitted. ``stream``: as in the forward.
    """
    lib = _bound or _bind()
    if stream is not None:
        return _on_stream(stream, qk_norm_rope_bwd, q, k, dq_out, dk_out, q_weight, k_weight, cos,
                          sin, positions, eps, interleaved, dq, dk, dq_weight, dk_weight,
                          weight_grads, workspace)
    if dq is None:
        dq = _dense_like(q)
    if dk is None:
        dk = _dense_like(k)
    own = (q.dtype,)
    dev, sizes, code, wcode, strides = _check_rope(
        (("q", q, own), ("k", k, own), ("dq_out", dq_out, (_torch.float32, q.dtype)),
         ("dk_out", dk_out, (dq_out.dtype,)), ("dq", dq, own), ("dk", dk, own)), q_weight,
        k_weight, cos, sin, positions)
    nbytes = 0
    if weight_grads:
        D = sizes[4]
        if dq_weight is None:
            dq_weight = _torch.empty(D, dtype=_torch.float32, device=q.device)
        if dk_weight is None:
            dk_weight = _torch.empty(D, dtype=_torch.float32, device=q.device)
        for w in (dq_weight, dk_weight):
            if w.dtype is not _torch.float32 or w.shape != (D,) or not w.is_contiguous() or \
                    w.get_device() != dev:
                raise ValueError("a weight's gradient must be a contiguous fp32 [D] tensor on "
                                 "q's device")
        if workspace is None:
            nbytes = norm_rope_bwd_workspace_bytes(sizes[0], sizes[1], D)
            workspace = _torch.empty(nbytes, dtype=_torch.uint8, device=q.device)
        else:
            nbytes = workspace.numel() * workspace.element_size()
            if workspace.get_device() != dev or not workspace.is_contiguous():
                raise ValueError("workspace must be a contiguous tensor on q's CUDA device")
    else:
        dq_weight = dk_weight = workspace = None
    st = _launch(dev, lib.nsa_qk_norm_rope_bwd, q.data_ptr(), k.data_ptr(),
                 dq_out.data_ptr(), dk_out.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                 _at(dq_weight), _at(dk_weight), _at(q_weight), _at(k_weight), _at(cos), _at(sin),
                 _at(positions), *sizes, eps, 1 if interleaved else 0, code, wcode,
                 _DTYPE_CODES[dq_out.dtype],
                 None if strides is None else strides.buffer_info()[0], _at(workspace), nbytes)
    if st != NSA_OK:
        raise NsaError(st, "nsa_qk_norm_rope_bwd")
    return dq, dk, dq_weight, dk_weight


class KvCache:
    """A paged cache of keys and values, as :func:`kv_append` fills it and
    :func:`paged_attn` reads it: the tensors, which stay the caller's.

    16 bits: ``k``, ``v`` fp16 or bf16 [pages, page_size, G, D]; strided views
    (of one tensor that holds both, say) with a contiguous last dimension and
    strides that are multiples of 8. 4 bits: ``k``, ``v`` uint8
    [pages, page_size, G, D/2] and ``k_scale``, ``v_scale`` bf16
    [pages, G, page_size, 2], all contiguous: byte i of a row holds the codes of
    entries 2i (lower four bits) and 2i + 1, an entry is low + step * code, and
    a scale is (step, low). page_size: a power of two from 16 to 1024.

    Sequences own pages through a page table, int32 [B, cols]: position p of
    sequence b is row p % page_size of page table[b, p // page_size]; an entry
    outside [0, pages), -1 say, is a page that the sequence does not have.
    """

    __slots__ = ("k", "v", "k_scale", "v_scale", "bits", "pages", "page_size", "kv_heads",
                 "head_dim", "_device", "_tail")

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if _torch is None:
            _bind()
        shape, dev = k.shape, k.get_device()
        if len(shape) != 4 or v.shape != shape or v.dtype is not k.dtype:
            raise ValueError("k and v must be alike, [pages, page_size, G, D]")
        pages, page, G, D = shape
        if k_scale is None and v_scale is None:
            if k.dtype not in _F16_KINDS:
                raise TypeError(f"a 16-bit cache must be fp16 or bf16, got {k.dtype}")
            a, b, c, last = k.stride()
            d, e, f, last_v = v.stride()
            if dev < 0 or v.get_device() != dev or last != 1 or last_v != 1:
                raise ValueError("k and v must be on one CUDA device, with a contiguous last "
                                 "dimension")
            # (the stride of a dimension of one is never used)
            if pages < 2:
                a = d = 0
            if G < 2:
                c = f = 0
            self._tail = (pages, page, a, b, c, d, e, f, 16)
            self.bits = 16
        elif k_scale is None or v_scale is None:
            raise ValueError("pass both scales (4 bits) or neither (16 bits)")
        else:
            if k.dtype is not _torch.uint8:
                raise TypeError(f"a 4-bit cache must be uint8, got {k.dtype}")
            bf16, scales = _torch.bfloat16, (pages, G, page, 2)
            if k_scale.dtype is not bf16 or v_scale.dtype is not bf16:
                raise TypeError("k_scale and v_scale must be bf16")
            if k_scale.shape != scales or v_scale.shape != scales:
                raise ValueError("k_scale and v_scale must be [pages, G, page_size, 2]")
            for t in (k, v, k_scale, v_scale):
                if t.get_device() != dev or dev < 0 or not t.is_contiguous():
                    raise ValueError("a 4-bit cache's tensors must be contiguous, on one CUDA "
                                     "device")
            D *= 2
            self._tail = (pages, page, 0, 0, 0, 0, 0, 0, 4)
            self.bits = 4
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.pages, self.page_size, self.kv_heads, self.head_dim = pages, page, G, D
        self._device = dev

    def _struct(self):
        """nsa_kv_cache: thirteen 8-byte fields."""
        if self.bits == 16:
            return array("Q", (self.k.data_ptr(), self.v.data_ptr(), 0, 0, *self._tail))
        return array("Q", (self.k.data_ptr(), self.v.data_ptr(), self.k_scale.data_ptr(),
                           self.v_scale.data_ptr(), *self._tail))


def kv_cache(pages: int, page_size: int, kv_heads: int, head_dim: int, dtype=None, bits: int = 16,
             device="cuda") -> KvCache:
    """An empty :class:`KvCache` of ``pages`` pages: ``dtype`` (bf16 by default)
    rows with ``bits`` 16, 4-bit rows with 4. What pages hold before tokens are
    stored is not defined, and is never seen."""
    import torch

    if bits == 16:
        dt = torch.bfloat16 if dtype is None else dtype
        shape = (pages, page_size, kv_heads, head_dim)
        return KvCache(*(torch.empty(shape, dtype=dt, device=device) for _ in range(2)))
    if bits != 4:
        raise ValueError(f"bits must be 16 or 4, got {bits}")
    shape = (pages, page_size, kv_heads, head_dim // 2)
    scale = (pages, kv_heads, page_size, 2)
    return KvCache(*(torch.empty(shape, dtype=torch.uint8, device=device) for _ in range(2)),
                   *(torch.empty(scale, dtype=torch.bfloat16, device=device) for _ in range(2)))


def _check_places(cache, page_table, positions, B, M, dev, need=False):
    """Checks of a cache's page table and positions; returns (columns, the
    stride of positions over the batch)."""
    if cache._device != dev:
        raise ValueError("the cache must be on the tensors' CUDA device")
    if page_table is None:
        raise ValueError("page_table must be [B, cols]")
    if page_table.dtype is not _torch.int32:
        raise TypeError(f"page_table must be int32, got {page_table.dtype}")
    ts = page_table.shape
    if len(ts) != 2 or ts[0] != B:
        raise ValueError("page_table must be [B, cols]")
    if page_table.get_device() != dev or not page_table.is_contiguous():
        raise ValueError("page_table must be a contiguous tensor on the cache's device")
    if positions is None:
        if need:
            raise ValueError("positions are needed: [M] or [B, M]")
        return ts[1], 0
    if positions.dtype is not _torch.int32:
        raise TypeError(f"positions must be int32, got {positions.dtype}")
    ps = positions.shape
    if ps != (B, M) and ps != (M,):
        raise ValueError("positions must be [M] or [B, M]")
    if positions.get_device() != dev or not positions.is_contiguous():
        raise ValueError("positions must be a contiguous tensor on the cache's device")
    return ts[1], M if len(ps) == 2 else 0


def kv_append(q, k, v, cache: KvCache, page_table, positions=None, q_weight=None, k_weight=None,
              cos=None, sin=None, eps: Optional[float] = 1e-6, interleaved: bool = False,
              q_out=None, *, stream=None):
    """Norm and rotation of new query and key heads, as :func:`qk_norm_rope`,
    with K and V stored in a paged cache (nsa_kv_append).

    q: fp16 or bf16 [B, M, H, D] (or None); k, v: [B, M, G, D] of q's dtype, and
    of the cache's where that has 16 bits; strided views are taken as in
    qk_norm_rope. ``page_table``: int32 [B, cols]. ``positions``, weights,
    tables, ``interleaved``: as in qk_norm_rope; ``eps`` None: no norm (and no
    weights), the rotation alone. Padding tokens, and tokens whose page the
    sequence does not have, are not stored. Two tokens of a call must not have
    the same place. Runs on torch's current stream, or on ``stream``. Returns
    q_out (None without q).
    """
    lib = _bound or _bind()
    if stream is not None:
        return _on_stream(stream, lambda k: kv_append(
            q, k, v, cache, page_table, positions, q_weight, k_weight, cos, sin, eps, interleaved,
            q_out), k)
    own = (k.dtype,)
    named = [("q", k[:, :, :0] if q is None else q, own), ("k", k, own)]
    if q is not None and q_out is not None:
        named.append(("q_out", q_out, own))
        named.append(("v", v, own))
    else:  # (places of q's shape and of k's take turns)
        named.append(named[0])
        named.append(("v", v, own))
    dev, sizes, code, wcode, strides = _check_rope(named, q_weight, k_weight, cos, sin, positions)
    B, M, H, G, D, R, rows, pstride = sizes
    if cache.kv_heads != G or cache.head_dim != D or (cache.bits == 16
                                                      and cache.k.dtype is not k.dtype):
        raise ValueError("the cache must have k's heads and entries, and with 16 bits its dtype")
    if eps is None:
        if q_weight is not None or k_weight is not None:
            raise ValueError("weights belong to the norm (eps)")
        eps = -1.0
    elif not eps >= 0:
        raise ValueError("eps must be >= 0, or None: no norm")
    cols, _ = _check_places(cache, page_table, positions, B, M, dev)
    new = H and q_out is None
    if strides is not None:  # (q, k, q_out, v) -> (k, v, q, q_out)
        s = strides
        strides = s[3:6] + s[9:12] + s[0:3] + \
            (array("q", (M * H * D, H * D, D)) if new else s[6:9])
    kv = cache._struct()
    if new:
        q_out = _torch.empty((B, M, H, D), dtype=q.dtype, device=q.device)
    st = _launch(dev, lib.nsa_kv_append, q.data_ptr() if H else None, k.data_ptr(), v.data_ptr(),
                 q_out.data_ptr() if H else None, kv.buffer_info()[0], page_table.data_ptr(),
                 _at(q_weight), _at(k_weight), _at(cos), _at(sin), _at(positions), B, M, H, G, D, R,
                 rows, pstride, cols, eps, 1 if interleaved else 0, code, wcode,
                 None if strides is None else strides.buffer_info()[0])
    if st != NSA_OK:
        raise NsaError(st, "nsa_kv_append")
    return q_out if H else None


def kv_read(cache: KvCache, page_table, positions, dtype=None, k_out=None, v_out=None, *,
            stream=None):
    """Rows of a paged cache as K and V (nsa_kv_read): [B, M, G, D] of the
    tokens at ``positions``, int32 [B, M] or [M], as :func:`sel_attn_fwd` and
    :func:`swa_fwd` take them. Zeros where a position is negative or its page
    one that the sequence does not have. ``dtype``: the cache's own with 16 bits;
    with 4 bits fp16 or bf16 (the default). Returns (k, v)."""
    lib = _bound or _bind()
    if stream is not None:
        return _on_stream(stream, lambda _: kv_read(cache, page_table, positions, dtype, k_out,
                                                    v_out), cache.k)
    if dtype is None:
        dtype = k_out.dtype if k_out is not None else \
            cache.k.dtype if cache.bits == 16 else _torch.bfloat16
    if dtype not in _F16_KINDS or (cache.bits == 16 and dtype is not cache.k.dtype):
        raise TypeError("dtype must be the cache's, or with 4 bits fp16 or bf16, got "
                        f"{dtype}")
    if page_table is None or page_table.dim() != 2:
        raise ValueError("page_table must be [B, cols]")
    if positions is None or not positions.dim():
        raise ValueError("positions are needed: [M] or [B, M]")
    B, M = page_table.shape[0], positions.shape[-1]
    dev = cache._device
    cols, pstride = _check_places(cache, page_table, positions, B, M, dev, need=True)
    shape = (B, M, cache.kv_heads, cache.head_dim)
    given = []
    if k_out is None:
        k_out = _torch.empty(shape, dtype=dtype, device=cache.k.device)
    else:
        given.append(("k_out", k_out))
    if v_out is None:
        v_out = _torch.empty_like(k_out)
    else:
        given.append(("v_out", v_out))
    for name, t in given:
        if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or \
                t.get_device() != dev:
            raise ValueError(f"{name} must be a contiguous {dtype} {shape} tensor on the cache's "
                             "device")
    kv = cache._struct()
    st = _launch(dev, lib.nsa_kv_read, kv.buffer_info()[0], page_table.data_ptr(),
                 positions.data_ptr(), k_out.data_ptr(), v_out.data_ptr(), B, M, cache.kv_heads,
                 cache.head_dim, pstride, cols, _DTYPE_CODES[dtype])
    if st != NSA_OK:
        raise NsaError(st, "nsa_kv_read")
    return k_out, v_out


def paged_attn_workspace_bytes(B, M, H, G, D, tokens, window=(-1, 0), sinks=0) -> int:
    """``tokens``: what a sequence's row of the page table can hold."""
    n = (_lib or load()).nsa_paged_attn_workspace_bytes(B, M, H, G, D, tokens, window[0], sinks)
    if n < 0:
        raise NsaError(int(n), "nsa_paged_attn_workspace_bytes")
    return n


def paged_attn(q, cache: KvCache, page_table, positions, window=(-1, 0), sinks: int = 0,
               scale: Optional[float] = None, out=None, lse=None, return_lse: bool = True,
               workspace=None, *, stream=None):
    """Attention of new tokens over a paged cache that holds their own keys and
    values too (nsa_paged_attn): a decoding step (M = 1), drafted tokens, or a
    piece of a prompt.

    q: fp16 or bf16 [B, M, H, D] (strided views as in :func:`kv_append`, but none
    that repeats rows by a stride of 0), of the cache's dtype where that has 16
    bits; ``page_table`` int32 [B, cols], ``positions`` int32 [B, M] or [M],
    negative: padding. The query at position p sees the keys j <= p of its sequence
    with j >= p - left or j < ``sinks`` (the first tokens, which stay visible behind
    the window), as far as the sequence has their pages; ``window`` = (left, 0), left
    negative: unbounded.
    Returns (O [B, M, H, D] of q's dtype, LSE fp32 [B, H, M] or None); O = 0 and
    LSE = -inf where a query sees nothing. ``workspace`` (CUDA uint8,
    paged_attn_workspace_bytes) is allocated when omitted and needed; calls that may
    overlap need one each. Runs on torch's current stream, or on ``stream``.
    """
    lib = _bound or _bind()
    if stream is not None:
        return _on_stream(stream, paged_attn, q, cache, page_table, positions, window, sinks, scale,
                          out, lse, return_lse, workspace)
    dt, qs = q.dtype, q.shape
    if dt not in _F16_KINDS:
        raise TypeError(f"q must be fp16 or bf16, got {dt}")
    if len(qs) != 4 or qs[3] != cache.head_dim:
        raise ValueError("q must be [B, M, H, D] with the cache's D")
    if cache.bits == 16 and cache.k.dtype is not dt:
        raise TypeError(f"q must be of the cache's dtype {cache.k.dtype}, got {dt}")
    B, M, H, D = qs
    dev = q.get_device()
    dense = q.is_contiguous()
    if dev < 0 or not (dense or q.stride(3) == 1):
        raise ValueError("q must be a CUDA tensor with a contiguous last dimension")
    cols, pstride = _check_places(cache, page_table, positions, B, M, dev, need=True)
    left, right = window
    if right != 0:
        raise ValueError("window must be (left, 0): the cache ends at the queries")
    if out is None:  # (empty_like takes 1.4 us less)
        out = _torch.empty_like(q) if dense else _torch.empty(qs, dtype=dt, device=q.device)
    elif out.dtype is not dt or out.shape != qs or not out.is_contiguous() or \
            out.get_device() != dev:
        raise ValueError(f"out must be a contiguous {dt} [B, M, H, D] tensor on q's device")
    if lse is None:
        if return_lse:
            lse = _torch.empty((B, H, M), dtype=_torch.float32, device=q.device)
    elif lse.dtype is not _torch.float32 or lse.shape != (B, H, M) or not lse.is_contiguous() or \
            lse.get_device() != dev:
        raise ValueError("lse must be a contiguous fp32 [B, H, M] tensor on q's device")
    strides = None
    if not dense:
        b, m, h, _ = q.stride()
        if (B > 1 and b == 0) or (M > 1 and m == 0) or (H > 1 and h == 0):
            raise ValueError("q must not repeat rows (a stride of 0)")
        strides = array("q", (b if B > 1 else 0, m if M > 1 else 0, h if H > 1 else 0))
    if workspace is None:
        tokens, nbytes = cols * cache.page_size, 0
        if tokens > 512:  # (0 up to there)
            nbytes = lib.nsa_paged_attn_workspace_bytes(B, M, H, cache.kv_heads, D, tokens, left,
                                                        sinks)
        if nbytes < 0:
            raise NsaError(nbytes, "nsa_paged_attn_workspace_bytes")
        if nbytes:
            workspace = _torch.empty(nbytes, dtype=_torch.uint8, device=q.device)
    else:
        nbytes = workspace.numel() * workspace.element_size()
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on q's CUDA device")
    kv = cache._struct()
    # scale: the ABI takes <= 0 for 1/sqrt(D)
    st = _launch(dev, lib.nsa_paged_attn, q.data_ptr(), kv.buffer_info()[0], page_table.data_ptr(),
                 positions.data_ptr(), out.data_ptr(), _at(lse), B, M, H, cache.kv_heads, D, pstride,
                 cols, left, sinks, 0.0 if scale is None else scale, _DTYPE_CODES[dt],
                 None if strides is None else strides.buffer_info()[0], _at(workspace), nbytes)
    if st != NSA_OK:
        raise NsaError(st, "nsa_paged_attn")
    return out, lse


def probe_l2_gather(k, v, g: int, block_size: int, ctas: int, warps_per_cta: int,
                    slots_per_warp: int, loads_per_warp: int, seed: int = 1, record=None,
                    stream=None, rows_per_box: int = 16) -> int:
    """Launch the gather-bandwidth probe (nsa_probe_l2_gather) on K, V
    [N, G, D] fp16 (one batch) and return the bytes it moves. ``record``: an
    int64 CUDA tensor [ctas, 3] for per-CTA (SM id, start ns, end ns), or
    None."""
    import torch

    lib = load()
    for name, t in (("k", k), ("v", v)):
        if t.dtype != torch.float16 or not t.is_cuda or not t.is_contiguous() or t.dim() != 3:
            raise ValueError(f"{name} must be a contiguous fp16 CUDA tensor [N, G, D]")
    if tuple(v.shape) != tuple(k.shape):
        raise ValueError("k and v must have the same shape")
    N, G, D = k.shape
    if record is not None and (record.dtype != torch.int64 or not record.is_cuda
                               or tuple(record.shape) != (ctas, 3)
                               or not record.is_contiguous()):
        raise ValueError("record must be a contiguous int64 CUDA tensor [ctas, 3]")
    if stream is None:
        stream = torch.cuda.current_stream(k.device)
    st = lib.nsa_probe_l2_gather(_ptr(k), _ptr(v), N, G, D, int(g), int(block_size), int(ctas),
                                 int(warps_per_cta), int(slots_per_warp), int(loads_per_warp),
                                 int(rows_per_box), int(seed) & 0xFFFFFFFF, _ptr(record),
                                 ctypes.c_void_p(stream.cuda_stream))
    if st != NSA_OK:
        raise NsaError(st, "nsa_probe_l2_gather")
    n = lib.nsa_probe_l2_gather_bytes(D, int(ctas), int(warps_per_cta), int(loads_per_warp),
                                      int(rows_per_box))
    if n < 0:
        raise NsaError(int(n), "nsa_probe_l2_gather_bytes")
    return int(n)


def probe_gather_rows(k, v, block_indices, block_size: int, ctas: int, warps_per_cta: int,
                      slots_per_warp: int, stream=None, extra_smem_bytes: int = 0) -> None:
    """Launch the index-driven gather probe (nsa_probe_gather_rows): the
    forward's copies for these rows alone. k, v: fp16 [B, N, G, D];
    block_indices: int32 [B, M, G, T], all contiguous on one CUDA device."""
    import torch

    lib = load()
    for name, t in (("k", k), ("v", v)):
        if t.dtype != torch.float16 or not t.is_cuda or not t.is_contiguous() or t.dim() != 4:
            raise ValueError(f"{name} must be a contiguous fp16 CUDA tensor [B, N, G, D]")
    if block_indices.dtype != torch.int32 or not block_indices.is_contiguous():
        raise ValueError("block_indices must be contiguous int32 [B, M, G, T]")
    B, N, G, D = k.shape
    Bi, M, Gi, T = block_indices.shape
    if (Bi, Gi) != (B, G) or tuple(v.shape) != tuple(k.shape):
        raise ValueError("shape mismatch: k/v [B, N, G, D], block_indices [B, M, G, T]")
    if stream is None:
        stream = torch.cuda.current_stream(k.device)
    st = lib.nsa_probe_gather_rows(_ptr(k), _ptr(v), _ptr(block_indices), B, M, N, G, D, T,
                                   int(block_size), int(ctas), int(warps_per_cta),
                                   int(slots_per_warp), int(extra_smem_bytes),
                                   ctypes.c_void_p(stream.cuda_stream))
    if st != NSA_OK:
        raise NsaError(st, "nsa_probe_gather_rows")


def probe_reduce_rows(buf, rows: int, stride: int, ctas: int, warps_per_cta: int,
                      iters_per_warp: int, seed: int = 1, stream=None) -> int:
    """Launch the reduction-rate probe (nsa_probe_reduce_rows) on an fp32
    CUDA tensor of at least rows * stride elements; returns the bytes it
    reduces. Adds zeros: the tensor's values are unchanged."""
    import torch

    lib = load()
    if buf.dtype != torch.float32 or not buf.is_cuda or buf.numel() < rows * stride:
        raise ValueError("buf must be an fp32 CUDA tensor of at least rows * stride elements")
    if stream is None:
        stream = torch.cuda.current_stream(buf.device)
    st = lib.nsa_probe_reduce_rows(_ptr(buf), int(rows), int(stride), int(ctas),
                                   int(warps_per_cta), int(iters_per_warp), int(seed) & 0xFFFFFFFF,
                                   ctypes.c_void_p(stream.cuda_stream))
    if st != NSA_OK:
        raise NsaError(st, "nsa_probe_reduce_rows")
    return int(ctas) * int(warps_per_cta) * int(iters_per_warp) * 4096
