"""Selective state space scan: binding of the ``kda_ssm_*`` entry points of ``include/kda.h``.

    y, hT = ssm_fwd(x, dt, A, B, C, D, dt_bias, h0, cu_seqlens)   # prompts, packed
    grads = ssm_bwd(x, dt, A, B, C, dy, D, dt_bias, h0, cu_seqlens, dh_T)
    y, h  = ssm_step(x, dt, A, B, C, h, D, dt_bias)               # one token per sequence, h in place
    y, st, h = ssm_conv_step(xbc, conv_weight, conv_state, dt, A, h, D, dt_bias, conv_bias)

Per head, with d_t = softplus(dt_t + dt_bias): h_t = exp(d_t A) h_{t-1} + d_t B_t^T x_t and
y_t = C_t h_t + D x_t.  x [T, H, P] and B, C [T, G, K] are bf16 or fp32 and may be slices of one
convolution's output; dt [T, H], the parameters A, D and dt_bias [H] and the states
[N, H, K, P] are fp32.  A group's H / G heads share its B and C.  The rules for strides,
outputs, workspaces and packed sequences are those of ``block.py``.
"""
from __future__ import annotations

import ctypes

import torch

from . import load_library
from .block import (_ACT, _apart, _code, _dims, _full, _given, _i32, _i64, _launch, _new, _p, _rank, _same_device, _seqs,
                    _size, _struct, _tokens, _workspace)

__all__ = ["ssm_fwd", "ssm_bwd", "ssm_step", "ssm_conv_step", "ssm_workspace_size", "ssm_conv_step_workspace_size"]


class _SsmDims(ctypes.Structure):
    _fields_ = [("num_seqs", _i32), ("heads", _i32), ("total_tokens", _i64), ("groups", _i32), ("state", _i32),
                ("width", _i32), ("dtype", _i32), ("softplus", _i32), ("reserved", _i32), ("x_stride", _i64),
                ("dt_stride", _i64), ("b_stride", _i64), ("c_stride", _i64), ("dy_stride", _i64)]


def _declare(lib):
    P, Z, D, I = ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(_SsmDims), ctypes.c_int
    for name, args in (("kda_ssm_fwd", [D] + [P] * 11 + [P, Z, P]), ("kda_ssm_bwd", [D] + [P] * 19 + [P, Z, P]),
                       ("kda_ssm_step", [D] + [P] * 10 + [P]), ("kda_ssm_conv_step", [D, I, I] + [P] * 12 + [P, Z, P]),
                       ("kda_ssm_workspace_size", [D, I, ctypes.POINTER(Z)]),
                       ("kda_ssm_conv_step_workspace_size", [D, ctypes.POINTER(Z)])):
        getattr(lib, name).restype = ctypes.c_int
        getattr(lib, name).argtypes = args


def _ssm_dims(x, dt, A, B, C, D, dt_bias, N, softplus, dy=None):
    T, H, P = shape = _rank(x, "x", 3)
    G, K = _rank(B, "B", 3)[1:]
    code = _code(x)
    xs = _tokens(x, "x", x.dtype, shape)
    bs = _tokens(B, "B", x.dtype, (T, G, K))
    cs = _tokens(C, "C", x.dtype, (T, G, K))
    ds = _tokens(dt, "dt", torch.float32, (T, H))
    ys = 0 if dy is None else _tokens(dy, "dy", x.dtype, shape)
    _full(_given(A, "A"), "A", torch.float32, (H,))
    _full(D, "D", torch.float32, (H,))
    _full(dt_bias, "dt_bias", torch.float32, (H,))
    return *_dims(_SsmDims, N, H, T, G, K, P, code, int(bool(softplus)), 0, xs, ds, bs, cs, ys), K


def ssm_fwd(x, dt, A, B, C, D=None, dt_bias=None, h0=None, cu_seqlens=None, *, softplus: bool = True,
            num_seqs: int | None = None, out=None, final_state=True, workspace=None):
    """The scan over packed sequences; returns (y [T, H, P], h_T [N, H, K, P] or None).

    D, dt_bias and h0 None: zeros.  softplus=False takes dt + dt_bias itself as the step,
    which must not be negative; A must not be positive.  cu_seqlens, num_seqs and
    final_state (True, False or a tensor to write, which must not be h0) are as for
    chunk_fwd.  workspace: a uint8 tensor of at least ssm_workspace_size bytes, or None to
    have one allocated."""
    lib = load_library()
    T, H, P = _rank(x, "x", 3)
    N = _seqs(cu_seqlens, num_seqs, T)
    d, ref, K = _ssm_dims(x, dt, A, B, C, D, dt_bias, N, softplus)
    _full(h0, "h0", torch.float32, (N, H, K, P))
    _full(out, "out", x.dtype, (T, H, P))
    given = isinstance(final_state, torch.Tensor)
    if given:
        _full(final_state, "final_state", torch.float32, (N, H, K, P))
    _same_device(x, dt=dt, A=A, B=B, C=C, D=D, dt_bias=dt_bias, h0=h0, cu_seqlens=cu_seqlens, out=out,
                 final_state=final_state if given else None, workspace=workspace)
    y = _new(x) if out is None else out
    hT = final_state if given else \
        torch.empty((N, H, K, P), dtype=torch.float32, device=x.device) if final_state else None
    ins = (x, dt, A, B, C, D, dt_bias, h0, cu_seqlens)
    for o in (out, hT if given else None):
        if o is not None:
            _apart(o, *ins, *(t for t in (out, hT) if t is not o))
    ws = _workspace("kda_ssm_workspace_size", d, (0,), workspace, x.device, *ins, out, hT)
    _launch(lib.kda_ssm_fwd, lib, x.device, (ref, _p(x), _p(dt), _p(A), _p(B), _p(C), _p(D), _p(dt_bias), _p(h0),
                                             _p(cu_seqlens), _p(y), _p(hT), _p(ws), ws.numel()))
    return y, hT


def ssm_bwd(x, dt, A, B, C, dy, D=None, dt_bias=None, h0=None, cu_seqlens=None, dh_T=None, *, softplus: bool = True,
            num_seqs: int | None = None, initial_state_grad=True, workspace=None):
    """Gradient of ssm_fwd for upstream derivatives dy [T, H, P] and dh_T [N, H, K, P] (None for
    zeros): a dict with "dx" [T, H, P], "dB" and "dC" [T, G, K] in x's dtype, "ddt" [T, H], "dA" [H],
    "dD" and "ddt_bias" [H] (None without D, dt_bias) and "dh0" [N, H, K, P] (None when
    initial_state_grad is False) in fp32.  workspace: at least
    ssm_workspace_size(backward=True) bytes."""
    lib = load_library()
    T, H, P = _rank(x, "x", 3)
    N = _seqs(cu_seqlens, num_seqs, T)
    d, ref, K = _ssm_dims(x, dt, A, B, C, D, dt_bias, N, softplus, _given(dy, "dy"))
    _full(h0, "h0", torch.float32, (N, H, K, P))
    _full(dh_T, "dh_T", torch.float32, (N, H, K, P))
    _same_device(x, dt=dt, A=A, B=B, C=C, dy=dy, D=D, dt_bias=dt_bias, h0=h0, cu_seqlens=cu_seqlens, dh_T=dh_T,
                 workspace=workspace)
    dev = x.device
    dx, dB, dC = _new(x), _new(B), _new(C)
    ddt = _new(dt)
    dA = torch.empty((H,), dtype=torch.float32, device=dev)
    dD = None if D is None else torch.empty_like(dA)
    db = None if dt_bias is None else torch.empty_like(dA)
    dh0 = torch.empty((N, H, K, P), dtype=torch.float32, device=dev) if initial_state_grad else None
    ws = _workspace("kda_ssm_workspace_size", d, (1,), workspace, dev, x, dt, A, B, C, dy, D, dt_bias, h0, cu_seqlens,
                    dh_T)
    _launch(lib.kda_ssm_bwd, lib, dev, (ref, _p(x), _p(dt), _p(A), _p(B), _p(C), _p(D), _p(dt_bias), _p(h0),
                                        _p(cu_seqlens), _p(dy), _p(dh_T), _p(dx), _p(ddt), _p(dA), _p(dB), _p(dC),
                                        _p(dD), _p(db), _p(dh0), _p(ws), ws.numel()))
    return {"dx": dx, "ddt": ddt, "dA": dA, "dB": dB, "dC": dC, "dD": dD, "ddt_bias": db, "dh0": dh0}


def ssm_workspace_size(x, B, *, num_seqs: int = 1, backward: bool = False):
    """Bytes of workspace ssm_fwd (or, backward=True, ssm_bwd) needs for the shapes of x and B."""
    T, H, P = _rank(x, "x", 3)
    G, K = _rank(B, "B", 3)[1:]
    return _size("kda_ssm_workspace_size",
                 _struct(_SsmDims, int(num_seqs), H, T, G, K, P, _code(x), 1, 0, 0, 0, 0, 0, 0), int(bool(backward)))


def ssm_step(x, dt, A, B, C, h, D=None, dt_bias=None, *, softplus: bool = True, out=None, h_out=None):
    """One token per sequence: x [N, H, P], dt [N, H], B, C [N, G, K], h [N, H, K, P] fp32, updated in
    place unless h_out is given; returns (y [N, H, P], state after).  A state that is updated in place is
    refused (KdaError) on any other tensor of the call, as one that is given apart is."""
    lib = load_library()
    N, H, P = _rank(x, "x", 3)
    d, ref, K = _ssm_dims(x, dt, A, B, C, D, dt_bias, N, softplus)
    _full(_given(h, "h"), "h", torch.float32, (N, H, K, P))
    _full(h_out, "h_out", torch.float32, (N, H, K, P))
    _full(out, "out", x.dtype, (N, H, P))
    _same_device(x, dt=dt, A=A, B=B, C=C, D=D, dt_bias=dt_bias, h=h, h_out=h_out, out=out)
    ho = h if h_out is None else h_out
    y = _new(x) if out is None else out
    ins = (x, dt, A, B, C, D, dt_bias)
    if out is not None:
        _apart(out, *ins, h, h_out)
    if h_out is not None and h_out is not h:
        _apart(h_out, *ins, *(() if h_out.data_ptr() == h.data_ptr() else (h,)))
    _launch(lib.kda_ssm_step, lib, x.device, (ref, _p(x), _p(dt), _p(A), _p(B), _p(C), _p(D), _p(dt_bias), _p(h),
                                              _p(ho), _p(y)))
    return y, ho


def _conv_step_dims(xbc, dt, h, softplus):
    N, channels = _rank(xbc, "xbc", 2)
    H, K, P = _rank(_given(h, "h"), "h", 4)[1:]
    rest = channels - H * P
    if K < 1:
        raise ValueError(f"h must have state rows (got {tuple(h.shape)})")
    if rest <= 0 or rest % (2 * K):
        raise ValueError(f"xbc has {channels} channels, which is not heads x width = {H} x {P} and 2 x groups x {K}")
    xs = _tokens(xbc, "xbc", xbc.dtype, (N, channels))
    ds = 0 if dt is None else _tokens(dt, "dt", torch.float32, (N, H))
    return _SsmDims, N, H, N, rest // (2 * K), K, P, _code(xbc, "xbc"), int(bool(softplus)), 0, xs, ds, 0, 0, 0


def ssm_conv_step(xbc, conv_weight, conv_state, dt, A, h, D=None, dt_bias=None, conv_bias=None, *, softplus: bool = True,
                  activation: str | None = "silu", out=None, conv_state_out=None, h_out=None, workspace=None):
    """One token per sequence through the layer's short convolution and the scan, the convolved
    values unrounded between them; returns (y [N, H, P], convolution state after, state after).

    xbc [N, H P + 2 G K] holds the projections of x, B and C in this order; conv_weight
    [channels, W] and conv_bias [channels] fp32 and conv_state [N, W - 1, channels] are as for
    conv_step, h [N, H, K, P] as for ssm_step.  Both states are updated in place unless
    conv_state_out or h_out is given, and then refused (KdaError) on each other or another tensor of
    the call.  workspace: at least ssm_conv_step_workspace_size
    bytes."""
    lib = load_library()
    dims = _conv_step_dims(xbc, dt, h, softplus)
    d, ref = _dims(*dims)
    N, H, K, P, channels = d.num_seqs, d.heads, d.state, d.width, xbc.shape[1]
    W = _rank(conv_weight, "conv_weight", 2)[1]
    if activation not in (None, "silu"):
        raise ValueError(f"activation must be None or 'silu' (got {activation!r})")
    _tokens(dt, "dt", torch.float32, (N, H))
    _full(conv_weight, "conv_weight", torch.float32, (channels, W))
    _full(conv_bias, "conv_bias", torch.float32, (channels,))
    states = (N, W - 1, channels)
    _full(_given(conv_state, "conv_state"), "conv_state", xbc.dtype, states)
    _full(conv_state_out, "conv_state_out", xbc.dtype, states)
    _full(_given(A, "A"), "A", torch.float32, (H,))
    _full(D, "D", torch.float32, (H,))
    _full(dt_bias, "dt_bias", torch.float32, (H,))
    _full(h, "h", torch.float32, (N, H, K, P))
    _full(h_out, "h_out", torch.float32, (N, H, K, P))
    _full(out, "out", xbc.dtype, (N, H, P))
    _same_device(xbc, conv_weight=conv_weight, conv_state=conv_state, dt=dt, A=A, h=h, D=D, dt_bias=dt_bias,
                 conv_bias=conv_bias, out=out, conv_state_out=conv_state_out, h_out=h_out, workspace=workspace)
    co = conv_state if conv_state_out is None else conv_state_out
    ho = h if h_out is None else h_out
    y = torch.empty((N, H, P), dtype=xbc.dtype, device=xbc.device) if out is None else out
    ins = (xbc, conv_weight, conv_bias, dt, A, D, dt_bias)
    if out is not None:
        _apart(out, *ins, conv_state, conv_state_out, h, h_out)
    if conv_state_out is not None and conv_state_out is not conv_state:
        _apart(conv_state_out, *ins, h, h_out, *(() if co.data_ptr() == conv_state.data_ptr() else (conv_state,)))
    if h_out is not None and h_out is not h:
        _apart(h_out, *ins, conv_state, *(() if ho.data_ptr() == h.data_ptr() else (h,)))
    ws = _workspace("kda_ssm_conv_step_workspace_size", d, (), workspace, xbc.device, *ins, conv_state, conv_state_out, h,
                    h_out, out)
    _launch(lib.kda_ssm_conv_step, lib, xbc.device,
            (ref, W, _ACT[activation], _p(xbc), _p(conv_weight), _p(conv_bias), _p(conv_state), _p(co), _p(dt), _p(A),
             _p(D), _p(dt_bias), _p(h), _p(ho), _p(y), _p(ws), ws.numel()))
    return y, co, ho


def ssm_conv_step_workspace_size(xbc, h):
    """Bytes of workspace ssm_conv_step needs for the shapes of xbc and h."""
    return _size("kda_ssm_conv_step_workspace_size", _struct(*_conv_step_dims(xbc, None, h, True)))
