"""ctypes binding of libcattn.so (include/cattn.h): the mixer operators that follow the
convolution, with the C ABI's names.

Like the convolution's binding, this module only checks and marshals arguments and allocates
outputs the caller does not pass.  Every step of the computation runs in the library's CUDA
kernels; there is no fallback.
"""
from __future__ import annotations

import ctypes
import re
from pathlib import Path

import torch

from . import _build
from .binding import (KernelDesc, _check, _device, _disjoint, _exact, _int32_vec, _ptr, _rows, _run,
                      _status, _stream, _wdt, _workspace, _WDTYPES, _cu)

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_INT = ctypes.c_int
_F32 = ctypes.c_float
_SZ = ctypes.c_size_t

CATTN_NORM_RMS = 0
CATTN_NORM_L2 = 1
_MODES = {"rms": CATTN_NORM_RMS, "l2": CATTN_NORM_L2}

_lib = None

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


def header_functions() -> list[str]:
    """Names of the functions include/cattn.h declares (CCONV_API ... name(...))."""
    text = (_build.INCLUDE / "cattn.h").read_text()
    return re.findall(r"CCONV_API\s+[\w\s\*]+?\b(\w+)\s*\(", text)


# ---------------------------------------------------------------------------------------
# norm of queries and keys with the position rotation
# ---------------------------------------------------------------------------------------

def _norm_args(q, k, wq, wk, cos, sin, positions, mode):
    """Checks shared by the norm's calls; returns (total, Hq, Hk, K, wdt, mode, P, R)."""
    _rows(q, "q", 3)
    _rows(k, "k", 3)
    total, Hq, K = q.shape
    if k.shape[0] != total or k.shape[2] != K:
        raise ValueError(f"k must be [{total}, Hk, {K}] like q, got shape {tuple(k.shape)}")
    wdt = 1
    for w, name in ((wq, "wq"), (wk, "wk")):
        if w is not None:
            if not isinstance(w, torch.Tensor) or w.dtype not in _WDTYPES:
                raise TypeError(f"{name} must be a float32 or bfloat16 tensor")
            _exact(w, (K,), w.dtype, name)
            wdt = _wdt(w)
    if wq is not None and wk is not None and wq.dtype != wk.dtype:
        raise TypeError("wq and wk must have the same dtype")
    if mode not in _MODES:
        raise ValueError(f"mode must be 'rms' or 'l2', got {mode!r}")
    P = R = 0
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin come together")
    if cos is not None:
        if not isinstance(cos, torch.Tensor) or cos.dim() != 2:
            raise ValueError("cos must be a [P, R/2] tensor")
        P, R = int(cos.shape[0]), 2 * int(cos.shape[1])
        _exact(cos, (P, R // 2), torch.float32, "cos")
        _exact(sin, (P, R // 2), torch.float32, "sin")
        if positions is not None:
            _int32_vec(positions, total, "positions")
        elif P < total:
            raise ValueError(f"without positions token t uses table row t: {P} rows for {total} tokens")
    elif positions is not None:
        raise ValueError("positions need the tables cos and sin")
    return total, Hq, k.shape[1], K, wdt, _MODES[mode], P, R


def cattn_qknorm_fwd(q: torch.Tensor, k: torch.Tensor, *, wq: torch.Tensor | None = None,
                     wk: torch.Tensor | None = None, cos: torch.Tensor | None = None,
                     sin: torch.Tensor | None = None, positions: torch.Tensor | None = None,
                     mode: str = "rms", eps: float = 1e-6, interleaved: bool = False,
                     yq: torch.Tensor | None = None, yk: torch.Tensor | None = None, stream=None):
    """Norm of each head of q [total, Hq, K] and k [total, Hk, K] (bf16), then the rotation of
    their first R channels by the tables cos, sin [P, R/2] (fp32; none: no rotation) at
    positions int32 [total] (none: row t).  Returns (yq, yk)."""
    total, Hq, Hk, K, wdt, m, P, R = _norm_args(q, k, wq, wk, cos, sin, positions, mode)
    outs = [("yq", yq, Hq), ("yk", yk, Hk)]
    for name, y, H in outs:
        if y is not None:
            _exact(y, (total, H, K), torch.bfloat16, name)
            _disjoint(((name, y),), (("q", q), ("k", k)))
    dev = _device(("q", "k", "wq", "wk", "cos", "sin", "positions", "yq", "yk"),
                  (q, k, wq, wk, cos, sin, positions, yq, yk))
    if yq is None:
        yq = torch.empty((total, Hq, K), dtype=torch.bfloat16, device=dev)
    if yk is None:
        yk = torch.empty((total, Hk, K), dtype=torch.bfloat16, device=dev)
    rc = _run(dev, load().cattn_qknorm_fwd, _ptr(q), q.stride(0), q.stride(1), _ptr(k), k.stride(0),
              k.stride(1), total, Hq, Hk, K, _ptr(wq), _ptr(wk), wdt, m, eps, _ptr(cos), _ptr(sin),
              P, R, int(bool(interleaved)), _ptr(positions), _ptr(yq), _ptr(yk),
              _stream(stream, dev))
    _check(rc, "cattn_qknorm_fwd")
    return yq, yk


def _bytes(call: str, dev, *sizes) -> int:
    n = _SZ(0)
    _check(_run(dev, getattr(load(), call), *sizes, ctypes.byref(n)), call)
    return int(n.value)


def _cuda(device) -> torch.device:
    return torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)


def cattn_qknorm_bwd_workspace_bytes(total: int, Hq: int, Hk: int, K: int, device=None) -> int:
    """Workspace cattn_qknorm_bwd needs on `device` (default: the current CUDA device)."""
    return _bytes("cattn_qknorm_bwd_workspace_bytes", _cuda(device), total, Hq, Hk, K)


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
    total, Hq, Hk, K, wdt, m, P, R = _norm_args(q, k, wq, wk, cos, sin, positions, mode)
    ins = (("q", q), ("k", k), ("dyq", dyq), ("dyk", dyk))
    for name, y, x in (("dyq", dyq, q), ("dyk", dyk, k)):
        _rows(y, name, 3)
        if y.shape != x.shape:
            raise ValueError(f"{name} must have shape {tuple(x.shape)}, got {tuple(y.shape)}")
    for name, y, H in (("dq", dq, Hq), ("dk", dk, Hk)):
        if y is not None:
            _exact(y, (total, H, K), torch.bfloat16, name)
            _disjoint(((name, y),), ins)
    for name, dw, w in (("dwq", dwq, wq), ("dwk", dwk, wk)):
        if dw is not None:
            if w is None:
                raise ValueError(f"{name} without its weight")
            _exact(dw, (K,), w.dtype, name)
    if workspace is not None:
        _workspace(workspace)
    dev = _device(("q", "k", "dyq", "dyk", "wq", "wk", "cos", "sin", "positions", "dq", "dk", "dwq",
                   "dwk", "workspace"),
                  (q, k, dyq, dyk, wq, wk, cos, sin, positions, dq, dk, dwq, dwk, workspace))
    if dq is None:
        dq = torch.empty((total, Hq, K), dtype=torch.bfloat16, device=dev)
    if dk is None:
        dk = torch.empty((total, Hk, K), dtype=torch.bfloat16, device=dev)
    if wq is not None and dwq is None:
        dwq = torch.empty(K, dtype=wq.dtype, device=dev)
    if wk is not None and dwk is None:
        dwk = torch.empty(K, dtype=wk.dtype, device=dev)
    if workspace is None and (dwq is not None or dwk is not None):
        workspace = torch.empty(cattn_qknorm_bwd_workspace_bytes(total, Hq, Hk, K, dev),
                                dtype=torch.uint8, device=dev)
    size = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = _run(dev, load().cattn_qknorm_bwd, _ptr(q), q.stride(0), q.stride(1), _ptr(k), k.stride(0),
              k.stride(1), _ptr(dyq), dyq.stride(0), dyq.stride(1), _ptr(dyk), dyk.stride(0),
              dyk.stride(1), total, Hq, Hk, K, _ptr(wq), _ptr(wk), wdt, m, eps, _ptr(cos),
              _ptr(sin), P, R, int(bool(interleaved)), _ptr(positions), _ptr(dq), _ptr(dk),
              _ptr(dwq), _ptr(dwk), _ptr(workspace), size, _stream(stream, dev))
    _check(rc, "cattn_qknorm_bwd")
    return dq, dk, dwq, dwk


# ---------------------------------------------------------------------------------------
# linear attention with a decay for each token and head
# ---------------------------------------------------------------------------------------

def _gates(g, rows: int, Hv: int):
    if not isinstance(g, torch.Tensor):
        raise TypeError(f"g must be a torch.Tensor, got {type(g).__name__}")
    if g.dtype != torch.float32:
        raise TypeError(f"g must be float32, got {g.dtype}")
    if tuple(g.shape) != (rows, Hv):
        raise ValueError(f"g must have shape {(rows, Hv)}, got {tuple(g.shape)}")


def _qkvg(q, k, v, g):
    """Checks shared by the linear calls; returns (rows, Hk, Hv, K, V)."""
    _rows(q, "q", 3)
    _rows(k, "k", 3)
    _rows(v, "v", 3)
    rows, Hk, K = q.shape
    if k.shape != q.shape:
        raise ValueError(f"k must have q's shape {tuple(q.shape)}, got {tuple(k.shape)}")
    if v.shape[0] != rows:
        raise ValueError(f"v must have q's {rows} rows, got {v.shape[0]}")
    Hv, V = v.shape[1:]
    if Hk < 1 or Hv < 1 or Hv % Hk:
        raise ValueError(f"the value heads ({Hv}) must be a multiple of the key heads ({Hk})")
    _gates(g, rows, Hv)
    return rows, Hk, Hv, K, V


def _states(t, name: str, Hv: int, K: int, V: int) -> int:
    """An fp32 state array [S, Hv, K, V], contiguous; returns S."""
    if not isinstance(t, torch.Tensor) or t.dim() != 4:
        raise ValueError(f"{name} must be a [S, {Hv}, {K}, {V}] tensor")
    _exact(t, (t.shape[0], Hv, K, V), torch.float32, name)
    return int(t.shape[0])


def _scale(scale, K: int) -> float:
    return K ** -0.5 if scale is None else float(scale)


def cattn_linear_fwd_workspace_bytes(total: int, nseq: int, Hk: int, Hv: int, K: int, V: int,
                                     device=None) -> int:
    """Workspace cattn_linear_fwd needs on `device` (default: the current CUDA device)."""
    return _bytes("cattn_linear_fwd_workspace_bytes", _cuda(device), total, nseq, Hk, Hv, K, V)


def cattn_linear_bwd_workspace_bytes(total: int, nseq: int, Hk: int, Hv: int, K: int, V: int,
                                     device=None) -> int:
    """Workspace cattn_linear_bwd needs on `device` (default: the current CUDA device)."""
    return _bytes("cattn_linear_bwd_workspace_bytes", _cuda(device), total, nseq, Hk, Hv, K, V)


def _work(workspace, call: str, dev, *sizes):
    if workspace is None:
        workspace = torch.empty(max(_bytes(call, dev, *sizes), 16), dtype=torch.uint8, device=dev)
    return workspace, workspace.numel() * workspace.element_size()


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
    int32 [nseq] sequence i's state is slot state_indices[i] and a status int32[2] is written.
    Returns (o, final_state or None, status or None)."""
    total, Hk, Hv, K, V = _qkvg(q, k, v, g)
    nseq = _cu(cu_seqlens)
    pools = []
    if initial_state is not None:
        pools.append(_states(initial_state, "initial_state", Hv, K, V))
    want_final = final_state is True
    if final_state is False or final_state is True:
        final_state = None
    if final_state is not None:
        pools.append(_states(final_state, "final_state", Hv, K, V))
    if state_indices is not None:
        _int32_vec(state_indices, nseq, "state_indices")
        if status is not None:
            _status(status)
    else:
        status = None
    if o is not None:
        _exact(o, (total, Hv, V), torch.bfloat16, "o")
    if o is not None or final_state is not None:
        _disjoint((("o", o), ("final_state", final_state)),
                  (("q", q), ("k", k), ("v", v), ("g", g)))
    if o is not None:
        _disjoint((("o", o),), (("initial_state", initial_state), ("final_state", final_state)))
    S = min(pools) if pools else nseq
    if want_final:
        S = min(S, nseq)
    if state_indices is None and (pools or want_final) and S < nseq:
        raise ValueError(f"without state_indices sequence i uses slot i: state arrays need at "
                         f"least nseq={nseq} slots")
    if workspace is not None:
        _workspace(workspace)
    dev = _device(("q", "k", "v", "g", "cu_seqlens", "initial_state", "final_state",
                   "state_indices", "status", "o", "workspace"),
                  (q, k, v, g, cu_seqlens, initial_state, final_state, state_indices, status, o,
                   workspace))
    if want_final:
        final_state = torch.empty((nseq, Hv, K, V), dtype=torch.float32, device=dev)
    if state_indices is not None and status is None:
        status = torch.empty(2, dtype=torch.int32, device=dev)
    if o is None:
        o = torch.empty((total, Hv, V), dtype=torch.bfloat16, device=dev)
    workspace, size = _work(workspace, "cattn_linear_fwd_workspace_bytes", dev, total, nseq, Hk, Hv,
                            K, V)
    rc = _run(dev, load().cattn_linear_fwd, _ptr(q), q.stride(0), q.stride(1), _ptr(k), k.stride(0),
              k.stride(1), _ptr(v), v.stride(0), v.stride(1), _ptr(g), g.stride(0), g.stride(1),
              total, Hk, Hv, K, V, _ptr(cu_seqlens), nseq, _scale(scale, K), _ptr(initial_state),
              _ptr(final_state), _ptr(state_indices), S, _ptr(status), _ptr(o), _ptr(workspace),
              size, _stream(stream, dev))
    _check(rc, "cattn_linear_fwd")
    return o, final_state, status


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
    total, Hk, Hv, K, V = _qkvg(q, k, v, g)
    nseq = _cu(cu_seqlens)
    _rows(do, "do", 3)
    if do.shape != v.shape:
        raise ValueError(f"do must have v's shape {tuple(v.shape)}, got {tuple(do.shape)}")
    S = nseq
    if initial_state is not None:
        S = _states(initial_state, "initial_state", Hv, K, V)
    if state_indices is not None:
        _int32_vec(state_indices, nseq, "state_indices")
        if status is None:
            raise ValueError("status (int32[2] on the device) is required with state_indices")
        _status(status)
    else:
        status = None
        if S < nseq:
            raise ValueError(f"without state_indices sequence i uses slot i: initial_state needs "
                             f"at least nseq={nseq} slots")
    if want_dinit is None:
        want_dinit = initial_state is not None or d_initial_state is not None
    if not want_dinit:
        d_initial_state = None
    given = (("dq", dq, (total, Hk, K), torch.bfloat16), ("dk", dk, (total, Hk, K), torch.bfloat16),
             ("dv", dv, (total, Hv, V), torch.bfloat16), ("dg", dg, (total, Hv), torch.float32),
             ("d_initial_state", d_initial_state, (nseq, Hv, K, V), torch.float32))
    for name, t, shape, dtype in given:
        if t is not None:
            _exact(t, shape, dtype, name)
            _disjoint(((name, t),), (("q", q), ("k", k), ("v", v), ("g", g), ("do", do),
                                     ("initial_state", initial_state)))
    if workspace is not None:
        _workspace(workspace)
    dev = _device(("q", "k", "v", "g", "do", "cu_seqlens", "initial_state", "state_indices",
                   "status", "dq", "dk", "dv", "dg", "d_initial_state", "workspace"),
                  (q, k, v, g, do, cu_seqlens, initial_state, state_indices, status, dq, dk, dv, dg,
                   d_initial_state, workspace))
    if dq is None:
        dq = torch.empty((total, Hk, K), dtype=torch.bfloat16, device=dev)
    if dk is None:
        dk = torch.empty((total, Hk, K), dtype=torch.bfloat16, device=dev)
    if dv is None:
        dv = torch.empty((total, Hv, V), dtype=torch.bfloat16, device=dev)
    if dg is None:
        dg = torch.empty((total, Hv), dtype=torch.float32, device=dev)
    if want_dinit and d_initial_state is None:
        d_initial_state = torch.empty((nseq, Hv, K, V), dtype=torch.float32, device=dev)
    workspace, size = _work(workspace, "cattn_linear_bwd_workspace_bytes", dev, total, nseq, Hk, Hv,
                            K, V)
    rc = _run(dev, load().cattn_linear_bwd, _ptr(q), q.stride(0), q.stride(1), _ptr(k), k.stride(0),
              k.stride(1), _ptr(v), v.stride(0), v.stride(1), _ptr(g), g.stride(0), g.stride(1),
              _ptr(do), do.stride(0), do.stride(1), total, Hk, Hv, K, V, _ptr(cu_seqlens), nseq,
              _scale(scale, K), _ptr(initial_state), _ptr(state_indices), S, _ptr(status), _ptr(dq),
              _ptr(dk), _ptr(dv), _ptr(dg), _ptr(d_initial_state), _ptr(workspace), size,
              _stream(stream, dev))
    _check(rc, "cattn_linear_bwd")
    return dq, dk, dv, dg, d_initial_state


def cattn_linear_update(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                        state: torch.Tensor, state_indices: torch.Tensor | None = None, *,
                        scale: float | None = None, pad_rows: bool = False,
                        o: torch.Tensor | None = None, status: torch.Tensor | None = None,
                        stream=None):
    """One token for each of N sequences: the recurrence on the pool state fp32 [S, Hv, K, V],
    updated in place unless status[0] reports CCONV_ERR_INDEX.  q, k [N, Hk, K], v [N, Hv, V]
    bf16; g [N, Hv] fp32.  pad_rows: index -1 marks a padding row (no state access, o row not
    written).  Returns (o [N, Hv, V], status int32[2] on the device)."""
    N, Hk, Hv, K, V = _qkvg(q, k, v, g)
    S = _states(state, "state", Hv, K, V)
    if state_indices is not None:
        _int32_vec(state_indices, N, "state_indices")
    elif S < N:
        raise ValueError(f"without state_indices row i uses slot i: state needs S >= N={N}")
    if o is not None:
        _exact(o, (N, Hv, V), torch.bfloat16, "o")
        _disjoint((("o", o),), (("q", q), ("k", k), ("v", v), ("g", g), ("state", state)))
    if status is not None:
        _status(status)
    dev = _device(("q", "k", "v", "g", "state", "state_indices", "o", "status"),
                  (q, k, v, g, state, state_indices, o, status))
    if o is None:
        o = torch.empty((N, Hv, V), dtype=torch.bfloat16, device=dev)
    if status is None:
        status = torch.empty(2, dtype=torch.int32, device=dev)
    rc = _run(dev, load().cattn_linear_update, _ptr(q), q.stride(0), q.stride(1), _ptr(k),
              k.stride(0), k.stride(1), _ptr(v), v.stride(0), v.stride(1), _ptr(g), g.stride(0),
              g.stride(1), N, Hk, Hv, K, V, _scale(scale, K), _ptr(state), S, _ptr(state_indices),
              int(bool(pad_rows)), _ptr(o), _ptr(status), _stream(stream, dev))
    _check(rc, "cattn_linear_update")
    return o, status


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
