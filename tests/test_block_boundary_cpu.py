"""Refusals of the operators around the state layer, on the host: status codes
of the C entry points (fake device addresses, never dereferenced) and the
binding's own checks (CPU)."""
import ctypes

import pytest
import torch

import kda_recurrent_state_amd as kda
from kda_recurrent_state_amd import block

OK, INVALID, UNSUPPORTED, MISALIGNED, HIP = 0, 1, 2, 3, 4
GOOD = 0x7F0000000000
ODD = GOOD + 1
OTHER = GOOD + (1 << 30)


@pytest.fixture(scope="module")
def lib():
    return kda.load_library()


def scan_dims(**kw):
    d = dict(num_seqs=2, channels=8, total_tokens=256, dtype=1, reserved=0, x_stride=0, log_a_stride=0, dy_stride=0)
    d.update(kw)
    return block._ScanDims(*d.values())


def conv_dims(**kw):
    d = dict(num_seqs=2, channels=8, total_tokens=64, dtype=1, width=4, activation=1, reserved=0, x_stride=0,
             dy_stride=0)
    d.update(kw)
    return block._ConvDims(*d.values())


def ng_dims(**kw):
    d = dict(tokens=4, heads=2, width=16, dtype=1, activation=2, eps=1e-6, reserved=0, x_stride=0, gate_stride=0,
             dy_stride=0)
    d.update(kw)
    return block._NormGateDims(*d.values())


def rn_dims(**kw):
    d = dict(tokens=4, width=16, dtype=1, residual_dtype=0, eps=1e-6, scale=1.0, reserved=0, x_stride=0,
             residual_stride=0, dy_stride=0, dresidual_stride=0)
    d.update(kw)
    return block._ResNormDims(*d.values())


ARGS = {  # after the dims: pointer arguments by name, in order
    "kda_scan_fwd": ("x log_a h0 cu y h_T states ws", True),
    "kda_scan_bwd": ("x log_a h0 cu states dy dh_T dx dlog_a dh0 ws", True),
    "kda_scan_step": ("x log_a h_in h_out y", False),
    "kda_conv_fwd": ("x weight bias state cu y state_T", False),
    "kda_conv_bwd": ("x weight bias state cu dy dstate_T dx dweight dbias dstate ws", True),
    "kda_conv_step": ("x weight bias state_in state_out y", False),
    "kda_norm_gate_fwd": ("x weight gate y", False),
    "kda_norm_gate_bwd": ("x weight gate dy dx dgate dweight ws", True),
    "kda_residual_norm_fwd": ("x residual weight cs residual_out y", False),
    "kda_residual_norm_bwd": ("x residual_out weight cs dy dres dx dresidual dweight dcs ws", True),
}


def call(lib, fn, dims, ws_bytes=1 << 40, **given):
    names, ws = ARGS[fn]
    ptrs = [given.get(n, GOOD + (i << 32)) for i, n in enumerate(names.split())]
    tail = ([ctypes.c_size_t(ws_bytes)] if ws else []) + [None]
    return getattr(lib, fn)(None if dims is None else ctypes.byref(dims), *ptrs, *tail)


DIMS = {"scan": scan_dims, "conv": conv_dims, "norm": ng_dims, "residual": rn_dims}


@pytest.mark.parametrize("fn", ARGS)
def test_null_dims(lib, fn):
    assert call(lib, fn, None) == INVALID and lib.kda_last_error().decode() == "dims is NULL"


CASES = [
    *[(f, dict(num_seqs=-1), {}, INVALID) for f in ("kda_scan_fwd", "kda_scan_bwd", "kda_conv_fwd", "kda_conv_bwd")],
    *[(f, dict(total_tokens=-1), {}, INVALID) for f in ("kda_scan_fwd", "kda_scan_bwd", "kda_conv_fwd", "kda_conv_bwd")],
    *[(f, dict(total_tokens=1 << 31), {}, INVALID) for f in ("kda_scan_fwd", "kda_conv_fwd")],
    *[(f, dict(channels=0), {}, INVALID) for f in ("kda_scan_fwd", "kda_scan_step", "kda_conv_bwd", "kda_conv_step")],
    *[(f, dict(channels=(1 << 20) + 1), {}, INVALID) for f in ("kda_scan_fwd", "kda_conv_fwd")],
    *[(f, dict(dtype=2), {}, INVALID) for f in ARGS],
    *[(f, dict(reserved=1), {}, INVALID) for f in ARGS],
    *[(f, dict(x_stride=3), {}, INVALID) for f in ARGS],
    *[(f, dict(x_stride=-8), {}, INVALID) for f in ARGS],
    *[(f, dict(x_stride=1 << 60), {}, INVALID) for f in ARGS],
    ("kda_scan_bwd", dict(dy_stride=7), {}, INVALID),
    ("kda_scan_fwd", dict(log_a_stride=7), {}, INVALID),
    ("kda_scan_fwd", dict(num_seqs=3), dict(cu=None), INVALID),       # 256 % 3
    ("kda_scan_fwd", dict(num_seqs=0), {}, INVALID),                  # tokens without a sequence
    ("kda_conv_bwd", dict(num_seqs=0), {}, INVALID),
    ("kda_scan_fwd", dict(num_seqs=0, total_tokens=0), {}, OK),
    ("kda_scan_bwd", dict(num_seqs=0, total_tokens=0), {}, OK),
    ("kda_conv_fwd", dict(num_seqs=0, total_tokens=0), {}, OK),
    ("kda_scan_step", dict(num_seqs=0, total_tokens=0), {}, OK),
    ("kda_conv_step", dict(num_seqs=0, total_tokens=0), {}, OK),
    ("kda_norm_gate_fwd", dict(tokens=0), {}, OK),
    ("kda_residual_norm_fwd", dict(tokens=0), {}, OK),
    ("kda_scan_step", {}, {}, INVALID),                               # 256 tokens, 2 sequences
    ("kda_conv_step", {}, {}, INVALID),
    ("kda_scan_fwd", {}, dict(x=None), INVALID),
    ("kda_scan_fwd", {}, dict(y=None), INVALID),
    ("kda_scan_fwd", {}, dict(x=ODD), MISALIGNED),
    ("kda_scan_fwd", {}, dict(log_a=GOOD + 2), MISALIGNED),
    ("kda_scan_fwd", {}, dict(h0=GOOD + 2), MISALIGNED),
    ("kda_scan_fwd", {}, dict(states=GOOD + 2), MISALIGNED),
    ("kda_scan_fwd", {}, dict(cu=GOOD + 2), MISALIGNED),
    ("kda_scan_fwd", {}, dict(h0=OTHER, h_T=OTHER), INVALID),
    ("kda_scan_fwd", {}, dict(ws=None), INVALID),
    ("kda_scan_fwd", {}, dict(ws_bytes=16), INVALID),
    ("kda_scan_fwd", {}, dict(ws=GOOD + 128), MISALIGNED),
    ("kda_scan_bwd", {}, dict(dy=None), INVALID),
    ("kda_scan_bwd", {}, dict(dlog_a=None), INVALID),
    ("kda_scan_bwd", {}, dict(dh0=OTHER, dh_T=OTHER), INVALID),
    ("kda_scan_bwd", {}, dict(ws_bytes=16), INVALID),
    ("kda_conv_fwd", dict(width=1), {}, UNSUPPORTED),
    ("kda_conv_bwd", dict(width=5), {}, UNSUPPORTED),
    ("kda_conv_step", dict(activation=2), {}, INVALID),
    ("kda_conv_fwd", {}, dict(weight=None), INVALID),
    ("kda_conv_fwd", {}, dict(state=OTHER, state_T=OTHER), INVALID),
    ("kda_conv_bwd", {}, dict(dstate=OTHER, dstate_T=OTHER), INVALID),
    ("kda_conv_bwd", {}, dict(ws=None), INVALID),
    ("kda_conv_bwd", {}, dict(dweight=GOOD + 2), MISALIGNED),
    ("kda_norm_gate_fwd", dict(width=0), {}, INVALID),
    ("kda_norm_gate_fwd", dict(width=8193), {}, UNSUPPORTED),
    ("kda_norm_gate_fwd", dict(heads=0), {}, INVALID),
    ("kda_norm_gate_fwd", dict(tokens=1 << 30, heads=4), {}, INVALID),
    ("kda_norm_gate_fwd", dict(eps=-1.0), {}, INVALID),
    ("kda_norm_gate_fwd", dict(eps=float("nan")), {}, INVALID),
    ("kda_norm_gate_fwd", dict(eps=float("inf")), {}, INVALID),
    ("kda_norm_gate_fwd", dict(activation=0), {}, INVALID),
    ("kda_norm_gate_fwd", dict(gate_stride=31), {}, INVALID),
    ("kda_norm_gate_fwd", dict(x_stride=64), dict(x=OTHER, y=OTHER), INVALID),  # in place over a strided x
    ("kda_norm_gate_bwd", {}, dict(dgate=None), INVALID),
    ("kda_norm_gate_bwd", {}, dict(gate=None), INVALID),
    ("kda_norm_gate_bwd", {}, dict(ws=None), INVALID),
    ("kda_norm_gate_bwd", dict(activation=7), {}, INVALID),
    ("kda_residual_norm_fwd", dict(width=8193), {}, UNSUPPORTED),
    ("kda_residual_norm_fwd", dict(dtype=0, residual_dtype=1), {}, UNSUPPORTED),
    ("kda_residual_norm_fwd", dict(residual_dtype=5), {}, INVALID),
    ("kda_residual_norm_fwd", dict(scale=float("inf")), {}, INVALID),
    ("kda_residual_norm_fwd", dict(residual_stride=17), dict(residual=OTHER, residual_out=OTHER), INVALID),
    ("kda_residual_norm_bwd", {}, dict(x=None), INVALID),            # needed for dchannel_scale
    ("kda_residual_norm_bwd", {}, dict(ws_bytes=4), INVALID),
    ("kda_residual_norm_bwd", dict(dresidual_stride=1), {}, INVALID),
]


@pytest.mark.parametrize("fn,change,given,expect", CASES)
def test_refusals(lib, fn, change, given, expect):
    d = DIMS[fn.split("_")[1]]()
    fields = [f[0] for f in d._fields_]
    if "num_seqs" not in fields and "num_seqs" in change:
        return
    for k, v in change.items():
        assert k in fields
        setattr(d, k, v)
    st = call(lib, fn, d, **given)
    assert st == expect, (st, lib.kda_last_error())


@pytest.mark.parametrize("fn", ["kda_scan_fwd", "kda_scan_bwd"])
def test_scan_larger_than_a_launch_is_refused(lib, fn):
    """ceil(T / 128) ceil(C / 64) workgroups of 512 threads, fewer than 2^32 - 64 * 512 threads in all."""
    first = (0xFFFFFFFF // 512 - 64) * 128 + 1
    for dims in (dict(total_tokens=first, channels=1), dict(total_tokens=first, channels=64),
                 dict(total_tokens=0x7FFF0000, channels=1), dict(total_tokens=first // 64, channels=64 * 65)):
        assert call(lib, fn, scan_dims(num_seqs=1, **dims)) == INVALID
        assert "too large" in lib.kda_last_error().decode()


def test_workspace_sizes(lib):
    n = ctypes.c_size_t(0)
    for T in (1, 64, 128, 129, 1000):
        tiles = -(-T // 128) if T > 128 else 0  # one tile passes no state on: no workspace
        assert lib.kda_scan_workspace_size(ctypes.byref(scan_dims(total_tokens=T)), 0, ctypes.byref(n)) == OK
        fwd = n.value
        assert lib.kda_scan_workspace_size(ctypes.byref(scan_dims(total_tokens=T)), 1, ctypes.byref(n)) == OK
        assert fwd >= tiles * 8 * 8 and fwd % 256 == 0 and (fwd > 0) == (T > 128)
        assert n.value >= fwd + -(-T // 64) * 8 * 4
    assert lib.kda_scan_workspace_size(ctypes.byref(scan_dims()), 0, None) == INVALID
    for fn, d in (("kda_conv_bwd_workspace_size", conv_dims()), ("kda_norm_gate_bwd_workspace_size", ng_dims()),
                  ("kda_residual_norm_bwd_workspace_size", rn_dims())):
        assert getattr(lib, fn)(ctypes.byref(d), ctypes.byref(n)) == OK and n.value > 0 and n.value % 256 == 0
        assert getattr(lib, fn)(ctypes.byref(d), None) == INVALID
        assert getattr(lib, fn)(None, ctypes.byref(n)) == INVALID


def t(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


BF = torch.bfloat16
BINDING = [
    # wrong types
    (TypeError, lambda: kda.scan_fwd(t(4, 3, dtype=torch.float16), t(4, 3))),
    (TypeError, lambda: kda.scan_fwd(t(4, 3), t(4, 3, dtype=BF))),
    (TypeError, lambda: kda.scan_fwd([1.0], t(4, 3))),
    (TypeError, lambda: kda.scan_fwd(t(4, 3), t(4, 3), cu_seqlens=torch.tensor([0, 4]))),
    (TypeError, lambda: kda.scan_fwd(t(4, 3), t(4, 3), cu_seqlens=[0, 4])),
    (TypeError, lambda: kda.scan_bwd(t(4, 3), t(4, 3), None)),
    (TypeError, lambda: kda.scan_step(t(4, 3), t(4, 3), None)),
    (TypeError, lambda: kda.conv_step(t(4, 3), t(3, 4), None)),
    (TypeError, lambda: kda.conv_fwd(t(4, 3), t(3, 4, dtype=BF))),
    (TypeError, lambda: kda.norm_gate_fwd(t(4, 2, 3), t(3), t(4, 2, 3, dtype=BF))),
    (TypeError, lambda: kda.residual_norm_fwd(t(4, 3), t(4, 3), None)),
    (TypeError, lambda: kda.residual_norm_bwd(None, t(4, 3), t(3), t(4, 3), channel_scale=t(3))),
    # wrong shapes
    (ValueError, lambda: kda.scan_fwd(t(4, 3), t(4, 2))),
    (ValueError, lambda: kda.scan_fwd(t(4, 3, 2), t(4, 3, 2))),
    (ValueError, lambda: kda.scan_fwd(t(4, 3), t(4, 3), t(2, 3))),
    (ValueError, lambda: kda.scan_fwd(t(4, 3), t(4, 3), num_seqs=-1)),
    (ValueError, lambda: kda.scan_fwd(t(4, 3), t(4, 3), cu_seqlens=torch.tensor([0, 4], dtype=torch.int32), num_seqs=2)),
    (ValueError, lambda: kda.scan_bwd(t(4, 3), t(4, 3), t(4, 3), states=t(2, 3))),
    (ValueError, lambda: kda.conv_fwd(t(4, 3), t(2, 4))),
    (ValueError, lambda: kda.conv_fwd(t(4, 3), t(3, 4), state=t(1, 4, 3))),
    (ValueError, lambda: kda.conv_fwd(t(4, 3), t(3, 4), activation="sigmoid")),
    (ValueError, lambda: kda.norm_gate_fwd(t(4, 2, 3), t(2))),
    (ValueError, lambda: kda.norm_gate_fwd(t(4, 2, 3), t(3), activation="relu")),
    (ValueError, lambda: kda.residual_norm_fwd(t(4, 3), t(4, 3), t(3), channel_scale=t(4))),
    # strides: transposed, overlapping (expanded) tokens, outputs that are not contiguous
    (ValueError, lambda: kda.scan_fwd(t(3, 4).t(), t(4, 3))),
    (ValueError, lambda: kda.scan_fwd(t(1, 3).expand(4, 3), t(4, 3))),
    (ValueError, lambda: kda.conv_bwd(t(4, 3), t(3, 4), t(1, 3).expand(4, 3))),
    (ValueError, lambda: kda.norm_gate_fwd(t(4, 2, 6)[:, :, :3], t(3))),
    (ValueError, lambda: kda.scan_fwd(t(4, 3), t(4, 3), out=t(4, 6)[:, :3])),
    # no CPU path
    (RuntimeError, lambda: kda.scan_fwd(t(4, 3), t(4, 3))),
    (RuntimeError, lambda: kda.scan_bwd(t(4, 3), t(4, 3), t(4, 3))),
    (RuntimeError, lambda: kda.scan_step(t(4, 3), t(4, 3), t(4, 3))),
    (RuntimeError, lambda: kda.conv_fwd(t(4, 3), t(3, 4))),
    (RuntimeError, lambda: kda.conv_bwd(t(4, 3), t(3, 4), t(4, 3))),
    (RuntimeError, lambda: kda.conv_step(t(4, 3), t(3, 4), t(4, 3, 3))),
    (RuntimeError, lambda: kda.norm_gate_fwd(t(4, 2, 3), t(3))),
    (RuntimeError, lambda: kda.norm_gate_bwd(t(4, 2, 3), t(3), t(4, 2, 3))),
    (RuntimeError, lambda: kda.residual_norm_fwd(t(4, 3), t(4, 3), t(3))),
    (RuntimeError, lambda: kda.residual_norm_bwd(t(4, 3), t(4, 3), t(3), t(4, 3))),
]


@pytest.mark.parametrize("i", range(len(BINDING)))
def test_binding_refusals(i):
    kind, fn = BINDING[i]
    with pytest.raises(kind):
        fn()


def test_overlapping_outputs_are_refused():
    base = t(8, 4)
    with pytest.raises(ValueError, match="overlaps"):
        block._apart(base[:4], base[3:7])
    with pytest.raises(ValueError, match="overlaps"):
        block._apart(base[2:4], base[:, :2])
    block._apart(base[:4], base[4:])
    block._apart(t(4, 4), base, None)
