"""Recurrent states kept in 8 bits: binding of the ``kda_state_cache_*`` entry points of ``include/kda.h``.

    codes, scales = state_cache_empty(num_slots, (H, dk, dv), torch.int8, device)
    state_cache_write(snapshots, codes, scales, slots)        # states [R, H, dk, dv] into their slots
    S0 = state_cache_read(codes, scales, slots)               # starting states of a later prefill

States are those of the state layer, of its snapshots or of the state space scan, float32 with any
number of dimensions; a state's last dimension is a row with one scale, the row's largest magnitude times
1/127 (int8) or 1/448 (float8_e4m3fn) in float32, and a code is the nearest of the format's values to the
quotient of value and scale, ties to even.  A row of zeros is kept exactly; one with an infinity or a NaN reads back as NaN.  A slot outside the
cache, such as -1, stands for no state: it is not written, and reads as zeros.  Where a call names a slot twice,
the last state stays.
"""
from __future__ import annotations

import ctypes

import torch

from . import load_library
from .block import _apart, _full, _i32, _i64, _launch, _p, _same_device, _struct

__all__ = ["state_cache_empty", "state_cache_write", "state_cache_read"]

_FORMAT = {torch.int8: 0, torch.float8_e4m3fn: 1}


class _CacheDims(ctypes.Structure):
    _fields_ = [("states", _i32), ("slots", _i32), ("rows", _i64), ("width", _i32), ("format", _i32),
                ("reserved", _i32)]


def _declare(lib):
    P, D = ctypes.c_void_p, ctypes.POINTER(_CacheDims)
    for name in ("kda_state_cache_write", "kda_state_cache_read"):
        getattr(lib, name).restype = ctypes.c_int
        getattr(lib, name).argtypes = [D, P, P, P, P, P]


def _cache(codes, scales, slots):
    """The cache's tensors checked: (dims of a state, format)."""
    if not isinstance(codes, torch.Tensor):
        raise TypeError("codes must be a torch.Tensor")
    if codes.dtype not in _FORMAT:
        raise TypeError(f"codes must be int8 or float8_e4m3fn (got {codes.dtype})")
    if codes.dim() < 2:
        raise ValueError(f"codes must be [slots, ..., width] (got {tuple(codes.shape)})")
    _full(codes, "codes", codes.dtype, codes.shape)
    if scales is None:
        raise TypeError("scales must be a torch.Tensor")
    _full(scales, "scales", torch.float32, codes.shape[:-1])
    if slots is not None:
        if not isinstance(slots, torch.Tensor) or slots.dtype is not torch.int32 or slots.dim() != 1 \
                or not slots.is_contiguous():
            raise TypeError("slots must be a contiguous 1-D int32 tensor")
    return codes.shape[1:], _FORMAT[codes.dtype]


def _rows(shape):
    n = 1
    for s in shape[:-1]:
        n *= s
    return n


def state_cache_empty(num_slots: int, shape, dtype=torch.int8, device="cuda"):
    """A cache of num_slots states of this shape, all zeros: (codes [num_slots, *shape] of dtype int8 or
    float8_e4m3fn, scales [num_slots, *shape[:-1]] float32)."""
    if dtype not in _FORMAT:
        raise TypeError(f"dtype must be int8 or float8_e4m3fn (got {dtype})")
    shape = tuple(shape)
    codes = torch.zeros((num_slots, *shape), dtype=torch.int8, device=device).view(dtype)
    return codes, torch.zeros((num_slots, *shape[:-1]), dtype=torch.float32, device=device)


def state_cache_write(states, codes, scales, slots=None):
    """Quantises states [R, *shape] float32 into the cache's slots (int32 [R] on the device; None: state r in
    slot r); returns (codes, scales)."""
    lib = load_library()
    shape, fmt = _cache(codes, scales, slots)
    if not isinstance(states, torch.Tensor):
        raise TypeError("states must be a torch.Tensor")
    R = states.shape[0] if states.dim() else 0
    _full(states, "states", torch.float32, (R, *shape))
    if slots is not None and slots.shape[0] != R:
        raise ValueError(f"slots holds {slots.shape[0]} entries for {R} states")
    _same_device(codes, scales=scales, states=states, slots=slots)
    _apart(codes, scales, states, slots)
    _apart(scales, states, slots)
    d = _struct(_CacheDims, R, codes.shape[0], _rows(shape), shape[-1], fmt, 0)
    _launch(lib.kda_state_cache_write, lib, codes.device, (ctypes.byref(d), _p(states), _p(slots), _p(codes), _p(scales)))
    return codes, scales


def state_cache_read(codes, scales, slots=None, *, out=None):
    """The states in these slots (int32 [R] on the device; None: all of them), [R, *shape] float32."""
    lib = load_library()
    shape, fmt = _cache(codes, scales, slots)
    R = codes.shape[0] if slots is None else slots.shape[0]
    _full(out, "out", torch.float32, (R, *shape))
    _same_device(codes, scales=scales, slots=slots, out=out)
    if out is None:
        out = torch.empty((R, *shape), dtype=torch.float32, device=codes.device)
    else:
        _apart(out, codes, scales, slots)
    d = _struct(_CacheDims, R, codes.shape[0], _rows(shape), shape[-1], fmt, 0)
    _launch(lib.kda_state_cache_read, lib, codes.device, (ctypes.byref(d), _p(codes), _p(scales), _p(slots), _p(out)))
    return out
