"""Gated half of a feed-forward block: binding of the ``kda_glu_*`` entry points of ``include/kda.h``.

    h = glu_fwd(x, w_gate, w_up)                       # act(x w_gate^T) * (x w_up^T)
    h, saved = glu_fwd_saved(x, w_gate, w_up)          # for training
    grads = glu_bwd(x, w_gate, w_up, dh, saved=saved)

x [T, D] and the weights [F, D] are bf16 or fp32, all of one type; the weights may be the halves of one
[2 F, D] tensor and x a slice of wider rows.  The activation of the gate is "silu", "sigmoid" or "gelu" (exact).
The rules for strides, outputs and workspaces are those of ``block.py``.
"""
from __future__ import annotations

import ctypes
from functools import lru_cache

import torch

from . import _check, load_library
from .block import (_apart, _bytes_apart, _code, _dims, _full, _given, _i32, _i64, _launch, _new, _p, _rank, _same_device,
                    _tokens)

__all__ = ["glu_fwd", "glu_fwd_saved", "glu_bwd", "glu_workspace_size"]

_GLU_ACT = {"silu": 1, "sigmoid": 2, "gelu": 3}


class _GluDims(ctypes.Structure):
    _fields_ = [("tokens", _i64), ("width", _i32), ("hidden", _i32), ("dtype", _i32), ("activation", _i32),
                ("x_stride", _i64), ("dh_stride", _i64)]


def _declare(lib):
    P, Z, D = ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(_GluDims)
    for name, args in (("kda_glu_fwd", [D] + [P] * 5 + [P, Z, P]), ("kda_glu_bwd", [D] + [P] * 8 + [P, Z, P]),
                       ("kda_glu_workspace_size", [D, P, P, P, ctypes.c_int, ctypes.POINTER(Z)])):
        getattr(lib, name).restype = ctypes.c_int
        getattr(lib, name).argtypes = args


def _glu_dims(x, w_gate, w_up, activation, dh=None):
    T, D = shape = _rank(x, "x", 2)
    F = _rank(w_gate, "w_gate", 2)[0]
    if activation not in _GLU_ACT:
        raise ValueError(f"activation must be 'silu', 'sigmoid' or 'gelu' (got {activation!r})")
    code = _code(x)
    xs = _tokens(x, "x", x.dtype, shape)
    _full(w_gate, "w_gate", x.dtype, (F, D))
    _full(_given(w_up, "w_up"), "w_up", x.dtype, (F, D))
    hs = 0 if dh is None else _tokens(dh, "dh", x.dtype, (T, F))
    return *_dims(_GluDims, T, D, F, code, _GLU_ACT[activation], xs, hs), (T, F)


@lru_cache(maxsize=4096)
def _glu_bytes(fields, x, wg, wu, backward):
    # the size depends on the addresses by whether 16 divides them
    lib = load_library()
    need = ctypes.c_size_t(0)
    d = _GluDims.from_buffer_copy(fields)
    _check(lib, lib.kda_glu_workspace_size(ctypes.byref(d), 256 + x, 256 + wg, 256 + wu, backward, ctypes.byref(need)))
    return need.value


def _glu_size(d, x, w_gate, w_up, backward):
    return _glu_bytes(bytes(d), x.data_ptr() % 16, w_gate.data_ptr() % 16, w_up.data_ptr() % 16, backward)


def _glu_workspace(d, x, w_gate, w_up, backward, workspace, *tensors):
    need = _glu_size(d, x, w_gate, w_up, backward)
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=x.device)
    if not isinstance(workspace, torch.Tensor) or workspace.dtype is not torch.uint8 or workspace.dim() != 1 \
            or not workspace.is_contiguous():
        raise TypeError("workspace must be a contiguous 1-D uint8 tensor")
    at = workspace.data_ptr()
    _bytes_apart("the workspace", at, at + min(need, workspace.numel()), (x, w_gate, w_up, *tensors))
    return workspace


def _glu(x, w_gate, w_up, activation, out, saved, workspace):
    lib = load_library()
    d, ref, shape = _glu_dims(x, w_gate, w_up, activation)
    _full(out, "out", x.dtype, shape)
    _full(saved, "saved", torch.float32, (2, *shape))
    _same_device(x, w_gate=w_gate, w_up=w_up, out=out, saved=saved, workspace=workspace)
    h = torch.empty(shape, dtype=x.dtype, device=x.device) if out is None else out
    for o in (out, saved):
        if o is not None:
            _apart(o, x, w_gate, w_up, *(t for t in (out, saved) if t is not o))
    ws = _glu_workspace(d, x, w_gate, w_up, 0, workspace, out, saved)
    _launch(lib.kda_glu_fwd, lib, x.device, (ref, _p(x), _p(w_gate), _p(w_up), _p(h), _p(saved), _p(ws), ws.numel()))
    return h


def glu_fwd(x, w_gate, w_up, *, activation: str = "silu", out=None, workspace=None):
    """h [T, F] = act(x w_gate^T) * (x w_up^T).  workspace: a uint8 tensor of at least
    glu_workspace_size bytes, or None to have one allocated."""
    return _glu(x, w_gate, w_up, activation, out, None, workspace)


def glu_fwd_saved(x, w_gate, w_up, *, activation: str = "silu", out=None, saved=None, workspace=None):
    """glu_fwd that keeps what glu_bwd needs of the forward: (h, saved [2, T, F] fp32), both products
    before the activation, unrounded."""
    if saved is None:
        T, F = _rank(x, "x", 2)[0], _rank(w_gate, "w_gate", 2)[0]
        saved = torch.empty((2, T, F), dtype=torch.float32, device=x.device)
    return _glu(x, w_gate, w_up, activation, out, saved, workspace), saved


def glu_bwd(x, w_gate, w_up, dh, *, activation: str = "silu", saved=None, input_grad=True, workspace=None):
    """Gradient of glu_fwd for dh [T, F]: a dict with "dx" [T, D] (None when input_grad is False),
    "dw_gate" and "dw_up" [F, D], in x's dtype.

    saved: as glu_fwd_saved returned it for the same inputs, or None to have both products computed
    again.  workspace: at least glu_workspace_size(backward=True) bytes."""
    lib = load_library()
    d, ref, shape = _glu_dims(x, w_gate, w_up, activation, _given(dh, "dh"))
    _full(saved, "saved", torch.float32, (2, *shape))
    _same_device(x, w_gate=w_gate, w_up=w_up, dh=dh, saved=saved, workspace=workspace)
    dx = _new(x) if input_grad else None
    dwg, dwu = _new(w_gate), _new(w_up)
    ws = _glu_workspace(d, x, w_gate, w_up, 1, workspace, dh, saved)
    _launch(lib.kda_glu_bwd, lib, x.device, (ref, _p(x), _p(w_gate), _p(w_up), _p(saved), _p(dh), _p(dx), _p(dwg),
                                             _p(dwu), _p(ws), ws.numel()))
    return {"dx": dx, "dw_gate": dwg, "dw_up": dwu}


def glu_workspace_size(x, w_gate, w_up, *, backward: bool = False):
    """Bytes of workspace glu_fwd (or, backward=True, glu_bwd) needs for these tensors (their shapes, and
    whether they lie at 16-byte addresses)."""
    return _glu_size(_glu_dims(x, w_gate, w_up, "silu")[0], x, w_gate, w_up, int(bool(backward)))
