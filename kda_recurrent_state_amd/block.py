"""Operators around the state layer: binding of the ``kda_scan_*``, ``kda_conv_*``,
``kda_norm_gate_*`` and ``kda_residual_norm_*`` entry points of ``include/kda.h``.

    y, r  = residual_norm_fwd(x, residual, w)                  # r = residual + scale x, y = rmsnorm(r) w
    q, st = conv_fwd(q_proj, w, bias, state, cu_seqlens)       # short causal convolution, SiLU
    h, hT = scan_fwd(x, log_a, h0, cu_seqlens)                 # h_t = exp(log_a_t) h_{t-1} + x_t
    y     = norm_gate_fwd(o, w, gate)                          # rmsnorm(o) w sigmoid(gate), per head

each with its gradient (``*_bwd``) and, where it keeps a state, one token per
sequence (``*_step``).  Tensors are bf16 or fp32; parameters (weight, bias,
channel_scale), log_a and the recurrence's states are fp32.  Inputs may be
slices of a fused projection: everything but the token stride must be
contiguous.  Outputs are contiguous, and allocated here unless given; one that is
given, or a given workspace's bytes, must not overlap another tensor of the call
(but for the updates in place that a call names).
Packed sequences are given as for ``chunk_fwd``; tokens at or past
``cu_seqlens[-1]`` are left alone, and so are their rows of the outputs.
"""
from __future__ import annotations

import ctypes
from functools import lru_cache

import torch

from . import KDA_BF16, KDA_F32, _check, load_library
from . import _same_device as _named_devices

__all__ = ["scan_fwd", "scan_fwd_states", "scan_bwd", "scan_step", "scan_workspace_size", "SCAN_STATE_EVERY",
           "conv_fwd", "conv_bwd", "conv_step", "conv_bwd_workspace_size",
           "norm_gate_fwd", "norm_gate_bwd", "norm_gate_bwd_workspace_size",
           "residual_norm_fwd", "residual_norm_bwd", "residual_norm_bwd_workspace_size"]

SCAN_STATE_EVERY = 64  # KDA_SCAN_STATE_EVERY
_ACT = {None: 0, "silu": 1, "sigmoid": 2}
_i32, _i64, _f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_float


class _ScanDims(ctypes.Structure):
    _fields_ = [("num_seqs", _i32), ("channels", _i32), ("total_tokens", _i64), ("dtype", _i32), ("reserved", _i32),
                ("x_stride", _i64), ("log_a_stride", _i64), ("dy_stride", _i64)]


class _ConvDims(ctypes.Structure):
    _fields_ = [("num_seqs", _i32), ("channels", _i32), ("total_tokens", _i64), ("dtype", _i32), ("width", _i32),
                ("activation", _i32), ("reserved", _i32), ("x_stride", _i64), ("dy_stride", _i64)]


class _NormGateDims(ctypes.Structure):
    _fields_ = [("tokens", _i64), ("heads", _i32), ("width", _i32), ("dtype", _i32), ("activation", _i32),
                ("eps", _f32), ("reserved", _i32), ("x_stride", _i64), ("gate_stride", _i64), ("dy_stride", _i64)]


class _ResNormDims(ctypes.Structure):
    _fields_ = [("tokens", _i64), ("width", _i32), ("dtype", _i32), ("residual_dtype", _i32), ("eps", _f32),
                ("scale", _f32), ("reserved", _i32), ("x_stride", _i64), ("residual_stride", _i64),
                ("dy_stride", _i64), ("dresidual_stride", _i64)]


def _declare(lib):
    """Argument types of the entry points bound here (called once, by load_library)."""
    P, Z = ctypes.c_void_p, ctypes.c_size_t
    for name, dims, before, workspace in (
            ("kda_scan_fwd", _ScanDims, 7, True), ("kda_scan_bwd", _ScanDims, 10, True),
            ("kda_scan_step", _ScanDims, 5, False),
            ("kda_conv_fwd", _ConvDims, 7, False), ("kda_conv_bwd", _ConvDims, 11, True),
            ("kda_conv_step", _ConvDims, 6, False),
            ("kda_norm_gate_fwd", _NormGateDims, 4, False), ("kda_norm_gate_bwd", _NormGateDims, 7, True),
            ("kda_residual_norm_fwd", _ResNormDims, 6, False), ("kda_residual_norm_bwd", _ResNormDims, 10, True)):
        fn = getattr(lib, name)
        fn.restype = ctypes.c_int
        fn.argtypes = [ctypes.POINTER(dims)] + [P] * before + ([P, Z] if workspace else []) + [P]
    for name, dims in (("kda_conv_bwd_workspace_size", _ConvDims), ("kda_norm_gate_bwd_workspace_size", _NormGateDims),
                       ("kda_residual_norm_bwd_workspace_size", _ResNormDims)):
        getattr(lib, name).restype = ctypes.c_int
        getattr(lib, name).argtypes = [ctypes.POINTER(dims), ctypes.POINTER(Z)]
    lib.kda_scan_workspace_size.restype = ctypes.c_int
    lib.kda_scan_workspace_size.argtypes = [ctypes.POINTER(_ScanDims), ctypes.c_int, ctypes.POINTER(Z)]


def _struct(kind, *fields):
    """A dims structure; ctypes itself takes an integer modulo its field's size."""
    for (name, of), v in zip(kind._fields_, fields):
        if of is _i32 and not -1 << 31 <= v < 1 << 31:
            raise ValueError(f"{name} = {v} does not fit 32 bits")
    return kind(*fields)


@lru_cache(maxsize=4096)
def _dims(kind, *fields):
    """A dims structure (only ever read) and a reference to it."""
    d = _struct(kind, *fields)
    return d, ctypes.byref(d)


def _code(t, name="x"):
    if t.dtype is torch.bfloat16:
        return KDA_BF16
    if t.dtype is torch.float32:
        return KDA_F32
    raise TypeError(f"{name} must be bfloat16 or float32 (got {t.dtype})")


def _tokens(t, name, dtype, shape):
    """A token tensor of this dtype and shape, contiguous but for the distance
    between its tokens, which is returned (in elements; 0: contiguous)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    if t.is_contiguous():
        return 0
    stride = t.stride()
    if len(stride) == 2 and stride[1] == 1 and stride[0] >= shape[1]:  # the usual slice
        return stride[0] if shape[0] > 1 else 0
    inner = 1
    for size, step in zip(reversed(shape[1:]), reversed(stride[1:])):
        if size > 1 and step != inner:
            raise ValueError(f"{name} must be contiguous within a token (strides {stride})")
        inner *= size
    if shape[0] > 1 and stride[0] < inner:
        raise ValueError(f"{name}'s tokens must not overlap (strides {stride})")
    return stride[0] if shape[0] > 1 else 0


def _full(t, name, dtype, shape):
    """A contiguous tensor of this dtype and shape, or None."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _given(t, name):
    if t is None:
        raise TypeError(f"{name} must be a torch.Tensor")
    return t


def _rank(t, name, ndim):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions (got {tuple(t.shape)})")
    return t.shape


def _seqs(cu_seqlens, num_seqs, T):
    """Number of sequences of a packed call."""
    if cu_seqlens is None:
        n = 1 if num_seqs is None else int(num_seqs)
        if n < 0:
            raise ValueError(f"num_seqs must not be negative (got {n})")
        return n
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dtype is not torch.int32 or cu_seqlens.dim() != 1 \
            or not cu_seqlens.is_contiguous() or cu_seqlens.shape[0] < 1:
        raise TypeError("cu_seqlens must be a contiguous 1-D int32 tensor [N + 1]")
    n = cu_seqlens.shape[0] - 1
    if num_seqs is not None and int(num_seqs) != n:
        raise ValueError(f"cu_seqlens holds {n} sequences, num_seqs says {int(num_seqs)}")
    return n


def _same_device(ref, **tensors):
    """Every tensor on ref's HIP device; the slower check says which is not."""
    dev = ref.device
    if dev.type != "cuda":
        _named_devices(ref)
    for t in tensors.values():
        if t is not None and t.device != dev:
            _named_devices(ref, **tensors)


def _touches(t, a, b):
    """Whether t, contiguous within its tokens, has a byte in [a, b)."""
    lo, size = t.data_ptr(), t.nbytes
    if not size or a >= b:
        return False
    if t.is_contiguous():
        return a < lo + size and lo < b
    tokens, step = t.shape[0], t.stride(0) * t.element_size()
    first = max(0, (a - lo - size // tokens) // step + 1)  # the first token that ends behind a
    return first < tokens and lo + first * step < b


def _apart(out, *inputs):
    """Refuses an output whose memory overlaps an input's."""
    at = out.data_ptr()
    _bytes_apart("an output", at, at + out.nbytes, inputs)


def _bytes_apart(what, a, b, tensors):
    for t in tensors:
        if t is not None and t.data_ptr() < b and _touches(t, a, b):
            raise ValueError(f"{what} overlaps another tensor of the call")


def _new(like):
    """An uninitialised contiguous tensor of like's shape (empty_like is the
    quicker call, and keeps the strides it is given)."""
    if like.is_contiguous():
        return torch.empty_like(like)
    return torch.empty(like.shape, dtype=like.dtype, device=like.device)


def _p(t):
    return None if t is None else t.data_ptr()


def _stream_of(i):
    return torch.cuda.current_stream(i).cuda_stream


# the same without the objects (1.9 us less) where torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _stream_of)


def _launch(fn, lib, device, args):
    """The entry point fn(args..., stream) on the tensors' device and its current
    stream (torch's current device is usually that one already)."""
    i = device.index
    if i == torch.cuda.current_device():
        status = fn(*args, _raw_stream(i))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _raw_stream(i))
    if status:
        _check(lib, status)


@lru_cache(maxsize=4096)
def _needed(name, kind, fields, more):
    lib = load_library()
    need = ctypes.c_size_t(0)
    d = kind.from_buffer_copy(fields)
    _check(lib, getattr(lib, name)(ctypes.byref(d), *more, ctypes.byref(need)))
    return need.value


def _workspace(name, dims, more, workspace, device, *tensors):
    """The caller's workspace, whose bytes that the call uses are none of its tensors', or
    one of the size that the entry point `name` says."""
    need = _needed(name, type(dims), bytes(dims), more)
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    if not isinstance(workspace, torch.Tensor) or workspace.dtype is not torch.uint8 or workspace.dim() != 1 \
            or not workspace.is_contiguous():
        raise TypeError("workspace must be a contiguous 1-D uint8 tensor")
    at = workspace.data_ptr()
    _bytes_apart("the workspace", at, at + min(need, workspace.numel()), tensors)
    return workspace


def _size(name, dims, *more):
    return _needed(name, type(dims), bytes(dims), more)


# ------------------------------------------------------------------ diagonal recurrence

def _scan_dims(x, log_a, N, dy=None):
    shape = x.shape
    code = _code(x)
    xs = 0 if x.is_contiguous() else _tokens(x, "x", x.dtype, shape)
    ls = _tokens(log_a, "log_a", torch.float32, shape)
    ds = 0 if dy is None else _tokens(dy, "dy", x.dtype, shape)
    return _dims(_ScanDims, N, shape[1], shape[0], code, 0, xs, ls, ds)


def _scan(x, log_a, h0, cu_seqlens, num_seqs, out, final_state, states, workspace):
    lib = load_library()
    T, C = _rank(x, "x", 2)
    N = _seqs(cu_seqlens, num_seqs, T)
    d, ref = _scan_dims(x, log_a, N)
    _full(h0, "h0", torch.float32, (N, C))
    _full(out, "out", x.dtype, (T, C))
    _full(states, "states", torch.float32, (-(-T // SCAN_STATE_EVERY), C))
    given = isinstance(final_state, torch.Tensor)
    if given:
        _full(final_state, "final_state", torch.float32, (N, C))
    _same_device(x, log_a=log_a, h0=h0, cu_seqlens=cu_seqlens, out=out, states=states,
                 final_state=final_state if given else None, workspace=workspace)
    y = _new(x) if out is None else out
    hT = final_state if given else torch.empty((N, C), dtype=torch.float32, device=x.device) if final_state else None
    for o in (out, hT if given else None, states):
        if o is not None:
            _apart(o, x, log_a, h0, cu_seqlens, *(t for t in (out, hT, states) if t is not o))
    ws = _workspace("kda_scan_workspace_size", d, (0,), workspace, x.device, x, log_a, h0, cu_seqlens, out, hT, states)
    _launch(lib.kda_scan_fwd, lib, x.device, (ref, _p(x), _p(log_a), _p(h0), _p(cu_seqlens), _p(y), _p(hT),
                                              _p(states), _p(ws), ws.numel()))
    return y, hT


def scan_fwd(x, log_a, h0=None, cu_seqlens=None, *, num_seqs: int | None = None, out=None, final_state=True,
             workspace=None):
    """Diagonal gated linear recurrence h_t = exp(log_a_t) h_{t-1} + x_t over packed
    sequences, per channel; returns (y, h_T or None), y_t = h_t.

    x [T, C] bf16 or fp32, log_a [T, C] fp32 (<= 0), h0 [N, C] fp32 or None for
    zeros, h_T [N, C] fp32.  cu_seqlens, num_seqs and final_state (True, False or a
    tensor to write, which must not be h0) are as for chunk_fwd.  workspace: a
    uint8 tensor of at least scan_workspace_size bytes, or None to have one
    allocated."""
    return _scan(x, log_a, h0, cu_seqlens, num_seqs, out, final_state, None, workspace)


def scan_fwd_states(x, log_a, h0=None, cu_seqlens=None, *, num_seqs: int | None = None, out=None, final_state=True,
                    states=None, workspace=None):
    """scan_fwd that keeps what scan_bwd needs of the forward: (y, h_T or None, states
    [ceil(T / 64), C] fp32), the state before every 64th token of the packed axis."""
    if states is None:
        T, C = _rank(x, "x", 2)
        states = torch.empty((-(-T // SCAN_STATE_EVERY), C), dtype=torch.float32, device=x.device)
    y, hT = _scan(x, log_a, h0, cu_seqlens, num_seqs, out, final_state, states, workspace)
    return y, hT, states


def scan_bwd(x, log_a, dy, h0=None, cu_seqlens=None, dh_T=None, *, num_seqs: int | None = None, states=None,
             initial_state_grad=True, workspace=None):
    """Gradient of scan_fwd for upstream derivatives dy [T, C] and dh_T [N, C] (None
    for zeros): a dict with "dx" (x's dtype), "dlog_a" [T, C] fp32 and "dh0" [N, C]
    fp32 (None when initial_state_grad is False).

    states: as scan_fwd_states returned them for the same inputs, or None to have
    them computed again.  workspace: at least scan_workspace_size(backward=True)
    bytes."""
    lib = load_library()
    T, C = _rank(x, "x", 2)
    N = _seqs(cu_seqlens, num_seqs, T)
    d, ref = _scan_dims(x, log_a, N, _given(dy, "dy"))
    _full(h0, "h0", torch.float32, (N, C))
    _full(dh_T, "dh_T", torch.float32, (N, C))
    _full(states, "states", torch.float32, (-(-T // SCAN_STATE_EVERY), C))
    _same_device(x, log_a=log_a, dy=dy, h0=h0, cu_seqlens=cu_seqlens, dh_T=dh_T, states=states, workspace=workspace)
    dev = x.device
    dx = _new(x)
    dla = _new(log_a)
    dh0 = torch.empty((N, C), dtype=torch.float32, device=dev) if initial_state_grad else None
    ws = _workspace("kda_scan_workspace_size", d, (1,), workspace, dev, x, log_a, dy, h0, cu_seqlens, dh_T, states)
    _launch(lib.kda_scan_bwd, lib, dev, (ref, _p(x), _p(log_a), _p(h0), _p(cu_seqlens), _p(states), _p(dy), _p(dh_T),
                                         _p(dx), _p(dla), _p(dh0), _p(ws), ws.numel()))
    return {"dx": dx, "dlog_a": dla, "dh0": dh0}


def scan_workspace_size(x, *, num_seqs: int = 1, backward: bool = False):
    """Bytes of workspace scan_fwd (or, backward=True, scan_bwd) needs for x's shape."""
    T, C = _rank(x, "x", 2)
    return _size("kda_scan_workspace_size", _struct(_ScanDims, int(num_seqs), C, T, _code(x), 0, 0, 0, 0),
                 int(bool(backward)))


def scan_step(x, log_a, h, *, out=None, h_out=None):
    """One token per sequence: x, log_a [N, C], h [N, C] fp32, updated in place unless
    h_out is given; returns (y, state after)."""
    lib = load_library()
    N, C = _rank(x, "x", 2)
    d, ref = _scan_dims(x, log_a, N)
    _full(_given(h, "h"), "h", torch.float32, (N, C))
    _full(h_out, "h_out", torch.float32, (N, C))
    _full(out, "out", x.dtype, (N, C))
    _same_device(x, log_a=log_a, h=h, h_out=h_out, out=out)
    ho = h if h_out is None else h_out
    y = _new(x) if out is None else out
    if out is not None:
        _apart(out, x, log_a, h, h_out)
    if h_out is not None and h_out is not h:
        _apart(h_out, x, log_a, *(() if h_out.data_ptr() == h.data_ptr() else (h,)))
    _launch(lib.kda_scan_step, lib, x.device, (ref, _p(x), _p(log_a), _p(h), _p(ho), _p(y)))
    return y, ho


# ------------------------------------------------------------------ short convolution

def _conv_dims(x, weight, bias, N, activation, dy=None):
    T, C = x.shape
    code = _code(x)
    W = _rank(weight, "weight", 2)[1]
    _full(weight, "weight", torch.float32, (C, W))
    _full(bias, "bias", torch.float32, (C,))
    if activation not in (None, "silu"):
        raise ValueError(f"activation must be None or 'silu' (got {activation!r})")
    xs = 0 if x.is_contiguous() else _tokens(x, "x", x.dtype, (T, C))
    ds = 0 if dy is None else _tokens(dy, "dy", x.dtype, (T, C))
    return *_dims(_ConvDims, N, C, T, code, W, _ACT[activation], 0, xs, ds), W


def conv_fwd(x, weight, bias=None, state=None, cu_seqlens=None, *, num_seqs: int | None = None,
             activation: str | None = "silu", out=None, final_state=True):
    """Causal depthwise convolution of W = 2, 3 or 4 taps over packed sequences, with an
    optional SiLU; returns (y, state_T or None).

    x [T, C], weight [C, W] fp32 (weight[:, -1] meets the token itself), bias [C]
    fp32 or None.  state [N, W - 1, C] in x's dtype holds the inputs before each
    sequence, oldest first (None: zeros); state_T the same after it.  final_state:
    True, False or a tensor to write, which must not be state."""
    lib = load_library()
    T, C = _rank(x, "x", 2)
    N = _seqs(cu_seqlens, num_seqs, T)
    d, ref, W = _conv_dims(x, weight, bias, N, activation)
    _full(state, "state", x.dtype, (N, W - 1, C))
    _full(out, "out", x.dtype, (T, C))
    given = isinstance(final_state, torch.Tensor)
    if given:
        _full(final_state, "final_state", x.dtype, (N, W - 1, C))
    _same_device(x, weight=weight, bias=bias, state=state, cu_seqlens=cu_seqlens, out=out,
                 final_state=final_state if given else None)
    y = _new(x) if out is None else out
    sT = final_state if given else torch.empty((N, W - 1, C), dtype=x.dtype, device=x.device) if final_state else None
    for o in (out, sT if given else None):
        if o is not None:
            _apart(o, x, weight, bias, state, cu_seqlens, *(t for t in (out, sT) if t is not o))
    _launch(lib.kda_conv_fwd, lib, x.device, (ref, _p(x), _p(weight), _p(bias), _p(state), _p(cu_seqlens),
                                              _p(y), _p(sT)))
    return y, sT


def conv_bwd(x, weight, dy, bias=None, state=None, cu_seqlens=None, dstate_T=None, *, num_seqs: int | None = None,
             activation: str | None = "silu", initial_state_grad=True, workspace=None):
    """Gradient of conv_fwd for upstream derivatives dy [T, C] and dstate_T [N, W - 1, C]
    (None for zeros): a dict with "dx" and "dstate" (x's dtype; "dstate" None when
    initial_state_grad is False), "dweight" [C, W] and "dbias" [C] fp32 (written also
    when bias is None).  workspace: at least conv_bwd_workspace_size bytes."""
    lib = load_library()
    T, C = _rank(x, "x", 2)
    N = _seqs(cu_seqlens, num_seqs, T)
    d, ref, W = _conv_dims(x, weight, bias, N, activation, _given(dy, "dy"))
    _full(state, "state", x.dtype, (N, W - 1, C))
    _full(dstate_T, "dstate_T", x.dtype, (N, W - 1, C))
    _same_device(x, weight=weight, dy=dy, bias=bias, state=state, cu_seqlens=cu_seqlens, dstate_T=dstate_T,
                 workspace=workspace)
    dev = x.device
    dx = _new(x)
    dw = _new(weight)
    db = torch.empty((C,), dtype=torch.float32, device=dev)
    ds = torch.empty((N, W - 1, C), dtype=x.dtype, device=dev) if initial_state_grad else None
    ws = _workspace("kda_conv_bwd_workspace_size", d, (), workspace, dev, x, weight, dy, bias, state, cu_seqlens,
                    dstate_T)
    _launch(lib.kda_conv_bwd, lib, dev, (ref, _p(x), _p(weight), _p(bias), _p(state), _p(cu_seqlens), _p(dy),
                                         _p(dstate_T), _p(dx), _p(dw), _p(db), _p(ds), _p(ws), ws.numel()))
    return {"dx": dx, "dweight": dw, "dbias": db, "dstate": ds}


def conv_bwd_workspace_size(x, width: int, *, num_seqs: int = 1):
    """Bytes of workspace conv_bwd needs for x's shape and `width` taps."""
    T, C = _rank(x, "x", 2)
    return _size("kda_conv_bwd_workspace_size",
                 _struct(_ConvDims, int(num_seqs), C, T, _code(x), int(width), 0, 0, 0, 0))


def conv_step(x, weight, state, bias=None, *, activation: str | None = "silu", out=None, state_out=None):
    """One token per sequence: x [N, C], state [N, W - 1, C], updated in place unless
    state_out is given; returns (y, state after)."""
    lib = load_library()
    N, C = _rank(x, "x", 2)
    d, ref, W = _conv_dims(x, weight, bias, N, activation)
    _full(_given(state, "state"), "state", x.dtype, (N, W - 1, C))
    _full(state_out, "state_out", x.dtype, (N, W - 1, C))
    _full(out, "out", x.dtype, (N, C))
    _same_device(x, weight=weight, state=state, bias=bias, state_out=state_out, out=out)
    so = state if state_out is None else state_out
    y = _new(x) if out is None else out
    if out is not None:
        _apart(out, x, weight, bias, state, state_out)
    if state_out is not None and state_out is not state:
        _apart(state_out, x, weight, bias, *(() if state_out.data_ptr() == state.data_ptr() else (state,)))
    _launch(lib.kda_conv_step, lib, x.device, (ref, _p(x), _p(weight), _p(bias), _p(state), _p(so), _p(y)))
    return y, so


# ------------------------------------------------------------------ norms

def _norm_gate_dims(x, weight, gate, activation, eps, dy=None):
    shape = _rank(x, "x", 3)
    T, H, D = shape
    if activation not in ("silu", "sigmoid"):
        raise ValueError(f"activation must be 'silu' or 'sigmoid' (got {activation!r})")
    _full(weight, "weight", torch.float32, (D,))
    xs = 0 if x.is_contiguous() else _tokens(x, "x", x.dtype, shape)
    gs = 0 if gate is None else _tokens(gate, "gate", x.dtype, shape)
    ds = 0 if dy is None else _tokens(dy, "dy", x.dtype, shape)
    return _dims(_NormGateDims, T, H, D, _code(x), _ACT[activation], float(eps), 0, xs, gs, ds)


def norm_gate_fwd(x, weight=None, gate=None, *, activation: str = "sigmoid", eps: float = 1e-6, out=None):
    """RMS norm of every head times a gate: x / sqrt(mean(x^2) + eps) * weight * act(gate).

    x, gate [T, H, D] (gate None: a plain RMS norm), weight [D] fp32 or None for ones,
    activation "sigmoid" or "silu" of the gate; returns y [T, H, D].  out may be x.  A
    norm over the whole width is H = 1."""
    lib = load_library()
    d, ref = _norm_gate_dims(x, weight, gate, activation, eps)
    _full(out, "out", x.dtype, x.shape)
    _same_device(x, weight=weight, gate=gate, out=out)
    y = _new(x) if out is None else out
    if out is not None:
        _apart(out, weight, gate, *(() if out.data_ptr() == x.data_ptr() and x.is_contiguous() else (x,)))
    _launch(lib.kda_norm_gate_fwd, lib, x.device, (ref, _p(x), _p(weight), _p(gate), _p(y)))
    return y


def norm_gate_bwd(x, weight, dy, gate=None, *, activation: str = "sigmoid", eps: float = 1e-6, workspace=None):
    """Gradient of norm_gate_fwd for dy [T, H, D]: a dict with "dx" and "dgate" (x's dtype;
    "dgate" None without a gate) and "dweight" [D] fp32 (None without a weight).
    workspace: at least norm_gate_bwd_workspace_size bytes (with a weight)."""
    lib = load_library()
    d, ref = _norm_gate_dims(x, weight, gate, activation, eps, _given(dy, "dy"))
    _same_device(x, weight=weight, dy=dy, gate=gate, workspace=workspace)
    dev = x.device
    dx = _new(x)
    dg = None if gate is None else _new(x)
    dw = None if weight is None else torch.empty(x.shape[2], dtype=torch.float32, device=dev)
    ws = None if dw is None else _workspace("kda_norm_gate_bwd_workspace_size", d, (), workspace, dev, x, weight, dy,
                                            gate)
    _launch(lib.kda_norm_gate_bwd, lib, dev, (ref, _p(x), _p(weight), _p(gate), _p(dy), _p(dx), _p(dg), _p(dw),
                                              _p(ws), 0 if ws is None else ws.numel()))
    return {"dx": dx, "dgate": dg, "dweight": dw}


def norm_gate_bwd_workspace_size(x):
    """Bytes of workspace norm_gate_bwd needs for x's shape."""
    T, H, D = _rank(x, "x", 3)
    return _size("kda_norm_gate_bwd_workspace_size",
                 _struct(_NormGateDims, T, H, D, _code(x), 2, 0.0, 0, 0, 0, 0))


def _res_norm_dims(x, res, weight, channel_scale, scale, eps, rname, dy=None, dres=None):
    shape = _rank(res, rname, 2)
    D = shape[1]
    like = x if x is not None else dy
    code, rcode = _code(like, "x" if x is not None else "dy"), _code(res, rname)
    _full(_given(weight, "weight"), "weight", torch.float32, (D,))
    _full(channel_scale, "channel_scale", torch.float32, (D,))
    xs = 0 if x is None else _tokens(x, "x", like.dtype, shape)
    rs = _tokens(res, rname, res.dtype, shape)
    ds = 0 if dy is None else _tokens(dy, "dy", like.dtype, shape)
    drs = 0 if dres is None else _tokens(dres, "dresidual_out", res.dtype, shape)
    return *_dims(_ResNormDims, shape[0], D, code, rcode, float(eps), float(scale), 0, xs, rs, ds, drs), like


def residual_norm_fwd(x, residual, weight, *, scale: float = 1.0, channel_scale=None, eps: float = 1e-6, out=None,
                      residual_out=None):
    """Residual sum and RMS norm in one pass: r = residual + scale * channel_scale * x and
    y = r / sqrt(mean(r^2) + eps) * weight; returns (y, r).

    x [T, D], residual [T, D] in x's dtype or fp32, weight and channel_scale [D] fp32
    (channel_scale None: ones).  y has x's dtype, r residual's; y is taken from the
    sum before its rounding.  residual_out may be residual."""
    lib = load_library()
    _rank(x, "x", 2)
    d, ref, _ = _res_norm_dims(x, residual, weight, channel_scale, scale, eps, "residual")
    _full(out, "out", x.dtype, x.shape)
    _full(residual_out, "residual_out", residual.dtype, x.shape)
    _same_device(x, residual=residual, weight=weight, channel_scale=channel_scale, out=out, residual_out=residual_out)
    y = _new(x) if out is None else out
    r = _new(residual) if residual_out is None else residual_out
    if out is not None:
        _apart(out, x, residual, weight, channel_scale, residual_out)
    if residual_out is not None:
        same = residual_out.data_ptr() == residual.data_ptr() and residual.is_contiguous()
        _apart(residual_out, x, weight, channel_scale, *(() if same else (residual,)))
    _launch(lib.kda_residual_norm_fwd, lib, x.device, (ref, _p(x), _p(residual), _p(weight),
                                                       _p(channel_scale), _p(r), _p(y)))
    return y, r


def residual_norm_bwd(x, residual_out, weight, dy, dresidual_out=None, *, scale: float = 1.0, channel_scale=None,
                      eps: float = 1e-6, workspace=None):
    """Gradient of residual_norm_fwd at the sum it returned (residual_out), for dy [T, D] and
    dresidual_out [T, D] (the stream's derivative from later blocks, None for zeros): a
    dict with "dx", "dresidual", "dweight" [D] fp32 and "dchannel_scale" [D] fp32 (None
    without channel_scale; x may be None then).  workspace: at least
    residual_norm_bwd_workspace_size bytes."""
    lib = load_library()
    if x is None and channel_scale is not None:
        raise TypeError("x is needed for the derivative of channel_scale")
    d, ref, like = _res_norm_dims(x, residual_out, weight, channel_scale, scale, eps, "residual_out", _given(dy, "dy"),
                             dresidual_out)
    _same_device(residual_out, x=x, weight=weight, channel_scale=channel_scale, dy=dy, dresidual_out=dresidual_out,
                 workspace=workspace)
    dev, shape = residual_out.device, residual_out.shape
    dx = _new(like)
    dr = _new(residual_out)
    dw = torch.empty(shape[1], dtype=torch.float32, device=dev)
    dc = None if channel_scale is None else torch.empty(shape[1], dtype=torch.float32, device=dev)
    ws = _workspace("kda_residual_norm_bwd_workspace_size", d, (), workspace, dev, x, residual_out, weight,
                    channel_scale, dy, dresidual_out)
    _launch(lib.kda_residual_norm_bwd, lib, dev, (ref, _p(x), _p(residual_out), _p(weight), _p(channel_scale), _p(dy),
                                                  _p(dresidual_out), _p(dx), _p(dr), _p(dw), _p(dc), _p(ws),
                                                  ws.numel()))
    return {"dx": dx, "dresidual": dr, "dweight": dw, "dchannel_scale": dc}


def residual_norm_bwd_workspace_size(x):
    """Bytes of workspace residual_norm_bwd needs for x's shape and dtype."""
    T, D = _rank(x, "x", 2)
    d = _struct(_ResNormDims, T, D, _code(x), _code(x), 0.0, 1.0, 0, 0, 0, 0, 0)
    return _size("kda_residual_norm_bwd_workspace_size", d)
