"""PyTorch binding of libcattn.so (include/cattn.h): the mixer operators that follow the
convolution, with the C ABI's names.

Like the convolution's binding, it only checks and marshals arguments and allocates outputs the
caller does not pass: every step of the computation runs in the library's CUDA kernels, and there
is no fallback.  The checks and the call are compiled (csrc/attn/py/attn_py.cpp, ``_cattn.so``);
this module holds the signatures.  load() gives the C ABI itself, through ctypes.

``stream`` (a torch stream or a raw handle) runs a call there, as under ``with
torch.cuda.stream(stream)``: the caller orders it after what made the inputs and before what reads
the results; tensors that the call makes for itself, the workspace among them, are safe by
themselves.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import re
from pathlib import Path

import torch

from . import _build
from .binding import CConvError, KernelDesc, _check, _run

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_INT = ctypes.c_int
_F32 = ctypes.c_float
_SZ = ctypes.c_size_t

CATTN_NORM_RMS = 0
CATTN_NORM_L2 = 1

_lib = None
_ext = None

_QK = [_P, _I64, _I64, _P, _I64, _I64]
_QKVG = _QK + [_P, _I64, _I64, _P, _I64, _I64]
_SIGNATURES = {
    "cattn_qknorm_fwd": _QK + [_I64] * 4 + [_P, _P, _INT, _INT, _F32, _P, _P, _I64, _I64, _INT, _P,
                                             _P, _P, _P],
    "cattn_qknorm_bwd_workspace_bytes": [_I64] * 4 + [ctypes.POINTER(_SZ)],
    "cattn_qknorm_bwd": _QK + _QK + [_I64] * 4 + [_P, _P, _INT, _INT, _F32, _P, _P, _I64, _I64,
                                                   _INT, _P, _P, _P, _P, _P, _P, _SZ, _P],
    "cattn_linear_fwd_workspace_bytes": [_I64] * 6 + [ctypes.POINTER(_SZ)],
    "cattn_linear_bwd_workspace_bytes": [_I64] * 6 + [ctypes.POINTER(_SZ)],
    "cattn_linear_fwd": _QKVG + [_I64] * 5 + [_P, _I64, _F32, _P, _P, _P, _I64, _P, _P, _P, _SZ, _P],
    "cattn_linear_bwd": _QKVG + [_P, _I64, _I64] + [_I64] * 5 + [_P, _I64, _F32, _P, _P, _I64, _P, _P,
                                                                 _P, _P, _P, _P, _P, _SZ, _P],
    "cattn_linear_update": _QKVG + [_I64] * 5 + [_F32, _P, _I64, _P, _INT, _P, _P, _P],
    "cattn_describe_begin": [],
    "cattn_describe_end": [ctypes.POINTER(KernelDesc), _INT, ctypes.POINTER(_INT)],
    "cattn_device_fault": [ctypes.POINTER(ctypes.c_int32)],
}


def lib_path() -> Path:
    return _build.ATTN_LIB


def load():
    """Load libcattn.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not _build.ATTN_LIB.exists():
        raise RuntimeError(
            f"{_build.ATTN_LIB} is missing: build the CUDA libraries first "
            "(python -m depthwise_causal_short_gb300._build, or __graft_entry__.build())")
    lib = ctypes.CDLL(str(_build.ATTN_LIB))
    for name, args in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, _INT
    _lib = lib
    return lib


def _calls():
    """The compiled binding (loaded once).  Raises if it has not been built."""
    global _ext
    if _ext is None:
        load()
        if not _build.ATTN_PY.exists():
            raise RuntimeError(f"{_build.ATTN_PY} is missing: build the libraries first")
        loader = importlib.machinery.ExtensionFileLoader("_cattn", str(_build.ATTN_PY))
        spec = importlib.util.spec_from_file_location("_cattn", str(_build.ATTN_PY), loader=loader)
        ext = importlib.util.module_from_spec(spec)
        loader.exec_module(ext)
        ext.set_error(CConvError)
        _ext = ext
    return _ext


def header_functions() -> list[str]:
    """Names of the functions include/cattn.h declares (CCONV_API ... name(...))."""
    text = (_build.INCLUDE / "cattn.h").read_text()
    return re.findall(r"CCONV_API\s+[\w\s\*]+?\b(\w+)\s*\(", text)


def _bytes(call: str, device, *sizes) -> int:
    n = _SZ(0)
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    _check(_run(dev, getattr(load(), call), *sizes, ctypes.byref(n)), call)
    return int(n.value)


# ---------------------------------------------------------------------------------------
# norm of queries and keys with the position rotation
# ---------------------------------------------------------------------------------------

def cattn_qknorm_fwd(q: torch.Tensor, k: torch.Tensor, *, wq: torch.Tensor | None = None,
                     wk: torch.Tensor | None = None, cos: torch.Tensor | None = None,
                     sin: torch.Tensor | None = None, positions: torch.Tensor | None = None,
                     mode: str = "rms", eps: float = 1e-6, interleaved: bool = False,
                     yq: torch.Tensor | None = None, yk: torch.Tensor | None = None, stream=None):
    """Norm of each head of q [total, Hq, K] and k [total, Hk, K] (bf16), then the rotation of
    their first R channels by the tables cos, sin [P, R/2] (fp32; none: no rotation) at
    positions int32 [total] (none: row t).  Returns (yq, yk)."""
    return _calls().qknorm_fwd(q, k, wq, wk, cos, sin, positions, mode, eps, interleaved, yq, yk, stream)


def cattn_qknorm_bwd_workspace_bytes(total: int, Hq: int, Hk: int, K: int, device=None) -> int:
    """Workspace cattn_qknorm_bwd needs on `device` (default: the current CUDA device)."""
    return _bytes("cattn_qknorm_bwd_workspace_bytes", device, total, Hq, Hk, K)


def cattn_qknorm_bwd(q: torch.Tensor, k: torch.Tensor, dyq: torch.Tensor, dyk: torch.Tensor, *,
                     wq: torch.Tensor | None = None, wk: torch.Tensor | None = None,
                     cos: torch.Tensor | None = None, sin: torch.Tensor | None = None,
                     positions: torch.Tensor | None = None, mode: str = "rms", eps: float = 1e-6,
                     interleaved: bool = False, dq: torch.Tensor | None = None,
                     dk: torch.Tensor | None = None, dwq: torch.Tensor | None = None,
                     dwk: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                     stream=None):
    """Gradient of cattn_qknorm_fwd: (dq, dk, dwq or None, dwk or None); a weight's gradient is
    computed when the weight is given."""
    return _calls().qknorm_bwd(q, k, wq, wk, cos, sin, positions, mode, eps, interleaved, dyq, dyk, dq, dk,
                               dwq, dwk, workspace, stream)


# ---------------------------------------------------------------------------------------
# linear attention with a decay for each token and head
# ---------------------------------------------------------------------------------------

def cattn_linear_fwd_workspace_bytes(total: int, nseq: int, Hk: int, Hv: int, K: int, V: int,
                                     device=None) -> int:
    """Workspace cattn_linear_fwd needs on `device` (default: the current CUDA device)."""
    return _bytes("cattn_linear_fwd_workspace_bytes", device, total, nseq, Hk, Hv, K, V)


def cattn_linear_bwd_workspace_bytes(total: int, nseq: int, Hk: int, Hv: int, K: int, V: int,
                                     device=None) -> int:
    """Workspace cattn_linear_bwd needs on `device` (default: the current CUDA device)."""
    return _bytes("cattn_linear_bwd_workspace_bytes", device, total, nseq, Hk, Hv, K, V)


def cattn_linear_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                     cu_seqlens: torch.Tensor, *, scale: float | None = None,
                     initial_state: torch.Tensor | None = None,
                     final_state: torch.Tensor | bool | None = None,
                     state_indices: torch.Tensor | None = None, status: torch.Tensor | None = None,
                     o: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                     stream=None):
    """Linear attention with decay over packed sequences: S_t = exp(g_t) S_{t-1} + k_t v_t^T,
    o_t = scale q_t^T S_t.  q, k [total, Hk, K], v [total, Hv, V] bf16; g [total, Hv] fp32 (any
    strides, e.g. expanded from [Hv]); cu_seqlens int32 [nseq+1]; scale defaults to K^-0.5.
    States fp32 [S, Hv, K, V]; final_state=True allocates [nseq, Hv, K, V]; with state_indices
    int32 [nseq] sequence i's state is slot state_indices[i] of both and a status int32[2] is written
    (a pool of more than nseq slots then wants a tensor for final_state, e.g. the pool itself).
    Returns (o, final_state or None, status or None)."""
    return _calls().linear_fwd(q, k, v, g, scale, cu_seqlens, initial_state, final_state, state_indices,
                               status, o, workspace, stream)


def cattn_linear_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                     do: torch.Tensor, cu_seqlens: torch.Tensor, *, scale: float | None = None,
                     initial_state: torch.Tensor | None = None,
                     state_indices: torch.Tensor | None = None, status: torch.Tensor | None = None,
                     want_dinit: bool | None = None, dq: torch.Tensor | None = None,
                     dk: torch.Tensor | None = None, dv: torch.Tensor | None = None,
                     dg: torch.Tensor | None = None, d_initial_state: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None, stream=None):
    """Gradient of cattn_linear_fwd's o: (dq, dk, dv, dg, d_initial_state or None).  The final
    states count as constants.  initial_state and state_indices as the forward read them
    (status, int32[2], is required with indices); d_initial_state is [nseq, Hv, K, V]."""
    return _calls().linear_bwd(q, k, v, g, scale, do, cu_seqlens, initial_state, state_indices, status,
                               want_dinit, dq, dk, dv, dg, d_initial_state, workspace, stream)


def cattn_linear_update(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                        state: torch.Tensor, state_indices: torch.Tensor | None = None, *,
                        scale: float | None = None, pad_rows: bool = False,
                        o: torch.Tensor | None = None, status: torch.Tensor | None = None,
                        stream=None):
    """One token for each of N sequences: the recurrence on the pool state fp32 [S, Hv, K, V],
    updated in place unless status[0] reports CCONV_ERR_INDEX.  q, k [N, Hk, K], v [N, Hv, V]
    bf16; g [N, Hv] fp32.  pad_rows: index -1 marks a padding row (no state access, o row not
    written).  Returns (o [N, Hv, V], status int32[2] on the device)."""
    return _calls().linear_update(q, k, v, g, scale, state, state_indices, pad_rows, o, status, stream)


def cattn_device_fault() -> int:
    v = ctypes.c_int32(0)
    _check(load().cattn_device_fault(ctypes.byref(v)), "cattn_device_fault")
    return int(v.value)


def attn_describe(fn) -> list[dict]:
    """The kernels fn() would launch through libcattn.so; see binding.describe."""
    lib = load()
    _check(lib.cattn_describe_begin(), "cattn_describe_begin")
    try:
        fn()
    finally:
        buf = (KernelDesc * 32)()
        n = ctypes.c_int(0)
        rc = lib.cattn_describe_end(buf, 32, ctypes.byref(n))
    _check(rc, "cattn_describe_end")
    return [{f: (getattr(d, f).decode() if f == "name" else getattr(d, f))
             for f, _ in KernelDesc._fields_} for d in buf[:min(n.value, 32)]]
