"""Refusals of the state space scan, the gated feed-forward products and the state cache, on the host: status
codes of the C entry points (fake device addresses, never dereferenced), the binding's own checks, sizes at
their limits and outputs that overlap other tensors (CPU)."""
import ctypes

import pytest
import torch

import kda_recurrent_state_amd as kda
from kda_recurrent_state_amd import block, feedforward, state_cache, statespace

OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3
GOOD = 0x7F0000000000


@pytest.fixture(scope="module")
def lib():
    return kda.load_library()


def ssm(**kw):
    d = dict(num_seqs=2, heads=4, total_tokens=256, groups=2, state=16, width=8, dtype=1, softplus=1, reserved=0,
             x_stride=0, dt_stride=0, b_stride=0, c_stride=0, dy_stride=0)
    d.update(kw)
    return statespace._SsmDims(*d.values())


def glu(**kw):
    d = dict(tokens=100, width=64, hidden=32, dtype=1, activation=1, x_stride=0, dh_stride=0)
    d.update(kw)
    return feedforward._GluDims(*d.values())


def cache(**kw):
    d = dict(states=3, slots=5, rows=8, width=16, format=0, reserved=0)
    d.update(kw)
    return state_cache._CacheDims(*d.values())


ARGS = {  # pointers after the dims (and plain integers), in order; whether a workspace follows
    "kda_ssm_fwd": ("x dt A B C D dt_bias h0 cu y h_T ws", True, ()),
    "kda_ssm_bwd": ("x dt A B C D dt_bias h0 cu dy dh_T dx ddt dA dB dC dD ddt_bias dh0 ws", True, ()),
    "kda_ssm_step": ("x dt A B C D dt_bias h_in h_out y", False, ()),
    "kda_ssm_conv_step": ("xbc conv_weight conv_bias conv_state_in conv_state_out dt A D dt_bias h_in h_out y ws", True, (4, 1)),
    "kda_glu_fwd": ("x w_gate w_up h saved ws", True, ()),
    "kda_glu_bwd": ("x w_gate w_up saved dh dx dw_gate dw_up ws", True, ()),
    "kda_state_cache_write": ("states slots codes scales", False, ()),
    "kda_state_cache_read": ("codes scales slots states", False, ()),
}
DIMS = {"ssm": ssm, "glu": glu, "state": cache}


def call(lib, fn, dims, ws_bytes=1 << 40, ints=None, **given):
    names, ws, plain = ARGS[fn]
    ptrs = [given.get(n, GOOD + (i << 32)) for i, n in enumerate(names.split())]
    tail = ([ctypes.c_size_t(ws_bytes)] if ws else []) + [None]
    return getattr(lib, fn)(None if dims is None else ctypes.byref(dims), *(plain if ints is None else ints), *ptrs, *tail)


def dims_of(fn, **kw):
    step = dict(num_seqs=7, total_tokens=7) if fn.endswith("step") else {}
    return DIMS[fn.split("_")[1]](**{**step, **kw})


@pytest.mark.parametrize("fn", ARGS)
def test_null_dims(lib, fn):
    assert call(lib, fn, None) == INVALID
    assert "dims is NULL" in lib.kda_last_error().decode()


NEEDED = {"kda_ssm_fwd": "x dt A B C y", "kda_ssm_bwd": "x dt A B C dy dx ddt dB dC", "kda_ssm_step": "x dt A B C h_in h_out y",
          "kda_ssm_conv_step": "xbc conv_weight conv_state_in conv_state_out dt A h_in h_out y", "kda_glu_fwd": "x w_gate w_up h",
          "kda_glu_bwd": "x w_gate w_up dh dw_gate dw_up", "kda_state_cache_write": "states codes scales",
          "kda_state_cache_read": "codes scales states"}


@pytest.mark.parametrize("fn,name", [(f, n) for f, s in NEEDED.items() for n in s.split()])
def test_null_pointers(lib, fn, name):
    assert call(lib, fn, dims_of(fn), **{name: None}) == INVALID
    assert name in lib.kda_last_error().decode()


@pytest.mark.parametrize("fn,name", [(f, n) for f in ARGS for n in ARGS[f][0].split() if n not in ("codes",)])
def test_misaligned_pointers(lib, fn, name):
    kw = dict(dtype=0) if fn == "kda_glu_fwd" and name == "ws" else {}  # bf16 of this width needs no workspace
    assert call(lib, fn, dims_of(fn, **kw), **{name: GOOD + 1}) == MISALIGNED
    assert ("workspace" if name == "ws" else "cu_seqlens" if name == "cu" else name) in lib.kda_last_error().decode()


BAD = [
    ("kda_ssm_fwd", dict(num_seqs=-1), INVALID), ("kda_ssm_fwd", dict(total_tokens=-1), INVALID),
    ("kda_ssm_fwd", dict(total_tokens=1 << 31), INVALID), ("kda_ssm_fwd", dict(heads=0), INVALID),
    ("kda_ssm_fwd", dict(heads=65537, groups=1), INVALID), ("kda_ssm_fwd", dict(groups=3), INVALID),
    ("kda_ssm_fwd", dict(groups=0), INVALID), ("kda_ssm_fwd", dict(state=0), INVALID),
    ("kda_ssm_fwd", dict(state=257), UNSUPPORTED), ("kda_ssm_fwd", dict(width=0), INVALID),
    ("kda_ssm_fwd", dict(width=8193), UNSUPPORTED), ("kda_ssm_fwd", dict(dtype=2), INVALID),
    ("kda_ssm_fwd", dict(softplus=2), INVALID), ("kda_ssm_fwd", dict(reserved=1), INVALID),
    ("kda_ssm_fwd", dict(x_stride=31), INVALID), ("kda_ssm_fwd", dict(dt_stride=3), INVALID),
    ("kda_ssm_fwd", dict(b_stride=31), INVALID), ("kda_ssm_fwd", dict(c_stride=-1), INVALID),
    ("kda_ssm_bwd", dict(dy_stride=31), INVALID), ("kda_ssm_fwd", dict(num_seqs=0), INVALID),
    ("kda_ssm_fwd", dict(num_seqs=1 << 30, heads=64), INVALID),
    ("kda_ssm_bwd", dict(num_seqs=1 << 24, total_tokens=1 << 24, heads=64), INVALID),
    ("kda_ssm_step", dict(total_tokens=8), INVALID), ("kda_ssm_conv_step", dict(total_tokens=8), INVALID),
    ("kda_ssm_step", dict(num_seqs=1 << 24, total_tokens=1 << 24), INVALID),
    ("kda_ssm_conv_step", dict(x_stride=95), INVALID),
    ("kda_glu_fwd", dict(tokens=-1), INVALID), ("kda_glu_fwd", dict(width=0), INVALID),
    ("kda_glu_fwd", dict(width=(1 << 20) + 1), INVALID), ("kda_glu_fwd", dict(hidden=0), INVALID),
    ("kda_glu_fwd", dict(hidden=(1 << 20) + 1), INVALID), ("kda_glu_fwd", dict(dtype=7), INVALID),
    ("kda_glu_fwd", dict(activation=0), INVALID), ("kda_glu_fwd", dict(activation=4), INVALID),
    ("kda_glu_fwd", dict(x_stride=63), INVALID), ("kda_glu_bwd", dict(dh_stride=31), INVALID),
    ("kda_glu_fwd", dict(tokens=1 << 30, hidden=1 << 20), INVALID),
    ("kda_state_cache_write", dict(states=-1), INVALID), ("kda_state_cache_write", dict(states=(1 << 20) + 1), INVALID),
    ("kda_state_cache_write", dict(slots=-1), INVALID), ("kda_state_cache_write", dict(rows=-1), INVALID),
    ("kda_state_cache_write", dict(rows=(1 << 40) + 1), INVALID), ("kda_state_cache_write", dict(width=0), INVALID),
    ("kda_state_cache_read", dict(width=8193), UNSUPPORTED), ("kda_state_cache_read", dict(format=2), INVALID),
    ("kda_state_cache_read", dict(reserved=1), INVALID),
    ("kda_state_cache_read", dict(slots=1 << 30, rows=1 << 30, width=8), INVALID),
    ("kda_state_cache_write", dict(slots=1, states=1 << 20, rows=1 << 40, width=8), INVALID),
]


@pytest.mark.parametrize("fn,kw,status", BAD, ids=str)
def test_bad_dims(lib, fn, kw, status):
    assert call(lib, fn, dims_of(fn, **kw)) == status
    assert lib.kda_last_error()


def test_other_refusals(lib):
    assert call(lib, "kda_ssm_fwd", ssm(total_tokens=255), cu=None) == INVALID  # not a multiple of the sequences
    assert call(lib, "kda_ssm_fwd", ssm(), h0=GOOD, h_T=GOOD) == INVALID
    assert call(lib, "kda_ssm_bwd", ssm(), dh_T=GOOD, dh0=GOOD) == INVALID
    assert call(lib, "kda_ssm_bwd", ssm(), h0=GOOD, dh0=GOOD) == INVALID
    assert call(lib, "kda_ssm_bwd", ssm(), ws_bytes=255) == INVALID
    assert call(lib, "kda_ssm_bwd", ssm(), ws=None) == INVALID
    for w, act in ((1, 1), (5, 1), (4, 2), (4, 3), (4, -1)):
        assert call(lib, "kda_ssm_conv_step", dims_of("kda_ssm_conv_step"), ints=(w, act)) in (INVALID, UNSUPPORTED)
    assert call(lib, "kda_ssm_conv_step", dims_of("kda_ssm_conv_step"), ws_bytes=0) == INVALID
    assert call(lib, "kda_glu_fwd", glu(dtype=0), ws_bytes=255) == INVALID
    assert call(lib, "kda_glu_bwd", glu(), ws_bytes=255) == INVALID
    assert call(lib, "kda_state_cache_write", cache(states=6), slots=None) == INVALID


def test_nothing_to_do(lib):
    """Calls without sequences, tokens or states are accepted whatever the pointers, and launch nothing."""
    none = {n: None for n in "x dt A B C D dt_bias h0 cu y h_T ws h_in h_out".split()}
    assert call(lib, "kda_ssm_fwd", ssm(num_seqs=0, total_tokens=0), ws_bytes=0, **none) == OK
    assert call(lib, "kda_ssm_step", ssm(num_seqs=0, total_tokens=0), **none) == OK
    assert call(lib, "kda_glu_fwd", glu(tokens=0), x=None, h=None, ws=None, ws_bytes=0) == OK
    assert call(lib, "kda_state_cache_write", cache(states=0), states=None, codes=None, scales=None, slots=None) == OK
    assert call(lib, "kda_state_cache_read", cache(rows=0), states=None, codes=None, scales=None) == OK


@pytest.mark.parametrize("backward", [0, 1])
def test_workspace_sizes(lib, backward):
    n = ctypes.c_size_t(0)
    size = lambda d: (lib.kda_ssm_workspace_size(ctypes.byref(d), backward, ctypes.byref(n)), n.value)
    for T in (0, 1, 63, 64, 65, 4096, 1 << 20):
        for H, G, K, P in ((1, 1, 1, 1), (32, 1, 128, 128), (10, 2, 40, 50), (64, 64, 256, 8192)):
            status, value = size(ssm(num_seqs=3, total_tokens=T, heads=H, groups=G, state=K, width=P))
            assert status == OK
            if backward and T:  # both kinds of states of every chunk are in it
                assert value >= 2 * (T // 64) * H * K * P * 4
    assert lib.kda_ssm_workspace_size(ctypes.byref(ssm()), backward, None) == INVALID
    # at the limits: refused, not wrapped around
    top = ssm(num_seqs=0x7fff0000, total_tokens=0x7fff0000, heads=65536, groups=1, state=256, width=8192)
    assert size(top)[0] == INVALID
    for T in (0, 1, 64, 65, 4097):
        for D, F, dt in ((64, 64, 1), (1, 1, 0), (1000, 2731, 0), (4096, 10240, 1)):
            d = glu(tokens=T, width=D, hidden=F, dtype=dt)
            assert lib.kda_glu_workspace_size(ctypes.byref(d), GOOD, GOOD, GOOD, backward, ctypes.byref(n)) == OK
            if backward:
                assert n.value >= 2 * T * F * (2 if dt else 6)
            # an address that is not 16-byte aligned costs a copy
            plain = n.value
            assert lib.kda_glu_workspace_size(ctypes.byref(d), GOOD + 4, GOOD, GOOD, backward, ctypes.byref(n)) == OK
            assert n.value >= plain


# ------------------------------------------------------------------ the binding

def f(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


T_, H_, G_, K_, P_, N_ = 40, 4, 2, 8, 6, 2
SSM = dict(x=lambda: f(T_, H_, P_), dt=lambda: f(T_, H_), A=lambda: f(H_), B=lambda: f(T_, G_, K_), C=lambda: f(T_, G_, K_))
OPT = dict(D=lambda: f(H_), dt_bias=lambda: f(H_), h0=lambda: f(N_, H_, K_, P_),
           cu_seqlens=lambda: torch.tensor([0, 10, T_], dtype=torch.int32))
STEP = dict(x=lambda: f(N_, H_, P_), dt=lambda: f(N_, H_), A=lambda: f(H_), B=lambda: f(N_, G_, K_), C=lambda: f(N_, G_, K_),
            h=lambda: f(N_, H_, K_, P_), D=lambda: f(H_), dt_bias=lambda: f(H_))
CH = H_ * P_ + 2 * G_ * K_
CONV = dict(xbc=lambda: f(N_, CH), conv_weight=lambda: f(CH, 4), conv_state=lambda: f(N_, 3, CH), dt=lambda: f(N_, H_),
            A=lambda: f(H_), h=lambda: f(N_, H_, K_, P_), D=lambda: f(H_), dt_bias=lambda: f(H_), conv_bias=lambda: f(CH))
GLU = dict(x=lambda: f(70, 32), w_gate=lambda: f(24, 32), w_up=lambda: f(24, 32))
CALLS = {"ssm_fwd": {**SSM, **OPT}, "ssm_bwd": {**SSM, "dy": lambda: f(T_, H_, P_), **OPT, "dh_T": lambda: f(N_, H_, K_, P_)},
         "ssm_step": STEP, "ssm_conv_step": CONV, "glu_fwd": GLU, "glu_fwd_saved": GLU,
         "glu_bwd": {**GLU, "dh": lambda: f(70, 24), "saved": lambda: f(2, 70, 24)}}
OUTS = {"ssm_fwd": dict(out=(T_, H_, P_), final_state=(N_, H_, K_, P_)), "ssm_step": dict(out=(N_, H_, P_), h_out=(N_, H_, K_, P_)),
        "ssm_conv_step": dict(out=(N_, H_, P_), conv_state_out=(N_, 3, CH), h_out=(N_, H_, K_, P_)), "glu_fwd": dict(out=(70, 24)),
        "glu_fwd_saved": dict(out=(70, 24), saved=(2, 70, 24))}
INPLACE = {("ssm_step", "h_out", "h"), ("ssm_conv_step", "h_out", "h"), ("ssm_conv_step", "conv_state_out", "conv_state")}


def args_of(fn):
    return {k: make() for k, make in CALLS[fn].items()}


@pytest.fixture()
def launched(monkeypatch):
    calls = []
    for mod in (block, statespace, feedforward, state_cache):
        monkeypatch.setattr(mod, "_same_device", lambda *a, **k: None)
        monkeypatch.setattr(mod, "_launch", lambda fn, lib, device, args: calls.append(fn.__name__))
    return calls


@pytest.mark.parametrize("fn", CALLS)
def test_no_cpu_path(fn):
    with pytest.raises(RuntimeError, match="HIP device"):
        getattr(kda, fn)(**args_of(fn))


@pytest.mark.parametrize("fn,name", [(fn, n) for fn in CALLS for n in CALLS[fn]])
def test_wrong_shapes_types_and_layouts(launched, fn, name):
    args = args_of(fn)
    getattr(kda, fn)(**args)
    assert len(launched) == 1
    good = args[name]
    wrong = [torch.zeros(*good.shape, 2), torch.zeros(3, *good.shape[1:]) if good.dim() > 1 else torch.zeros(good.shape[0] + 1),
             good.to(torch.float64), good.to(torch.float16)]
    if name == "x" and fn in ("glu_fwd", "glu_fwd_saved"):
        wrong.pop(1)  # x alone says how many tokens there are
    if good.dim() > 1 and good.shape[-1] > 1:
        wide = torch.zeros(*good.shape[:-1], 2 * good.shape[-1], dtype=good.dtype)
        wrong.append(wide[..., ::2])  # holes within a token
    for w in wrong:
        with pytest.raises((TypeError, ValueError)):
            getattr(kda, fn)(**{**args, name: w})
    with pytest.raises((TypeError, AttributeError)):
        getattr(kda, fn)(**{**args, name: [1.0]})
    assert len(launched) == 1


def within(t, shape):
    """A float32 tensor of this shape in t's memory, from its first byte."""
    n = torch.empty(shape).nbytes
    big = torch.zeros(t.nbytes + n, dtype=torch.uint8)
    return big[:n].view(torch.float32).view(shape), big[:t.nbytes].view(t.dtype).view(t.shape)


@pytest.mark.parametrize("fn,out,inp", [(fn, o, i) for fn in OUTS for o in OUTS[fn] for i in CALLS[fn]
                                        if (fn, o, i) not in INPLACE])
def test_an_output_over_an_input(launched, fn, out, inp):
    args = args_of(fn)
    given = {k: f(*s) for k, s in OUTS[fn].items()}
    getattr(kda, fn)(**args, **given)
    assert len(launched) == 1
    given[out], args[inp] = within(args[inp], OUTS[fn][out])
    if inp == "cu_seqlens":
        args[inp].copy_(OPT[inp]())
    with pytest.raises(ValueError, match="overlaps"):
        getattr(kda, fn)(**args, **given)
    assert len(launched) == 1


@pytest.mark.parametrize("fn,name", [(fn, n) for fn in ("ssm_bwd", "ssm_conv_step", "glu_bwd") for n in CALLS[fn]])
def test_a_workspace_over_a_tensor(launched, fn, name):
    args = args_of(fn)
    nbytes = 1 << 21
    getattr(kda, fn)(**args, workspace=torch.zeros(nbytes, dtype=torch.uint8))
    assert len(launched) == 1
    big = torch.zeros(nbytes, dtype=torch.uint8)
    t = args[name]
    args[name] = big[:t.nbytes].view(t.dtype).view(t.shape)
    if name == "cu_seqlens":
        args[name].copy_(OPT[name]())
    with pytest.raises(ValueError, match="overlaps"):
        getattr(kda, fn)(**args, workspace=big)
    assert len(launched) == 1


def test_update_in_place(launched):
    a = args_of("ssm_conv_step")
    y, cs, h = kda.ssm_conv_step(**a)
    assert cs is a["conv_state"] and h is a["h"]
    kda.ssm_conv_step(**a, conv_state_out=a["conv_state"], h_out=a["h"])
    s = args_of("ssm_step")
    assert kda.ssm_step(**s)[1] is s["h"]
    kda.ssm_step(**s, h_out=s["h"].view(s["h"].shape))
    assert len(launched) == 4


def test_other_arguments(launched):
    a = args_of("ssm_conv_step")
    for act in ("sigmoid", "gelu", 1):
        with pytest.raises(ValueError, match="activation"):
            kda.ssm_conv_step(**a, activation=act)
    for xbc in (f(N_, H_ * P_), f(N_, CH + 1)):
        with pytest.raises(ValueError, match="channels"):
            kda.ssm_conv_step(**{**a, "xbc": xbc})
    g = args_of("glu_fwd")
    for act in (None, "relu", 1):
        with pytest.raises(ValueError, match="activation"):
            kda.glu_fwd(**g, activation=act)
    with pytest.raises(TypeError):
        kda.glu_fwd(**g, workspace=f(100))
    s = args_of("ssm_fwd")
    with pytest.raises(ValueError, match="num_seqs"):
        kda.ssm_fwd(**s, num_seqs=3)
    assert not launched


def test_state_cache_arguments(launched):
    codes, scales = kda.state_cache_empty(5, (2, 3, 4), torch.int8, "cpu")
    x, slots = f(2, 2, 3, 4), torch.tensor([1, 3], dtype=torch.int32)
    kda.state_cache_write(x, codes, scales, slots)
    kda.state_cache_read(codes, scales, slots, out=f(2, 2, 3, 4))
    assert launched == ["kda_state_cache_write", "kda_state_cache_read"]
    bad = [lambda: kda.state_cache_write(f(2, 2, 3, 5), codes, scales, slots),
           lambda: kda.state_cache_write(x.double(), codes, scales, slots),
           lambda: kda.state_cache_write(x, codes.to(torch.int16), scales, slots),
           lambda: kda.state_cache_write(x, codes, scales[:4], slots),
           lambda: kda.state_cache_write(x, codes, scales.double(), slots),
           lambda: kda.state_cache_write(x, codes, None, slots),
           lambda: kda.state_cache_write(x, codes, scales, slots.long()),
           lambda: kda.state_cache_write(x, codes, scales, slots[:1]),
           lambda: kda.state_cache_write(x, codes[..., ::2], scales, slots),
           lambda: kda.state_cache_read(codes, scales, slots, out=f(3, 2, 3, 4)),
           lambda: kda.state_cache_read([1], scales, slots),
           lambda: kda.state_cache_empty(3, (2, 4), torch.float16, "cpu")]
    for b in bad:
        with pytest.raises((TypeError, ValueError)):
            b()
    # tensors in each other's memory
    buf = torch.zeros(4096, dtype=torch.uint8)
    codes2 = buf[:120].view(torch.int8).view(5, 2, 3, 4)
    for over in (lambda: kda.state_cache_write(buf[:192].view(torch.float32).view(2, 2, 3, 4), codes2, scales, slots),
                 lambda: kda.state_cache_write(x, codes2, buf[100:220].view(torch.float32).view(5, 2, 3), slots),
                 lambda: kda.state_cache_read(codes2, scales, slots, out=buf[64:256].view(torch.float32).view(2, 2, 3, 4))):
        with pytest.raises(ValueError, match="overlaps"):
            over()
    assert len(launched) == 2


def test_sizes_past_32_bits():
    m = lambda *s: torch.empty(*s, device="meta")
    wrap = 1 << 32
    for name, fn in (("heads", lambda: kda.ssm_workspace_size(m(1, wrap + 2, 4), m(1, 1, 4))),
                     ("width", lambda: kda.ssm_workspace_size(m(1, 2, wrap + 4), m(1, 1, 4))),
                     ("state", lambda: kda.ssm_workspace_size(m(1, 2, 4), m(1, 1, wrap + 4))),
                     ("num_seqs", lambda: kda.ssm_workspace_size(m(1, 2, 4), m(1, 1, 4), num_seqs=wrap + 1)),
                     ("hidden", lambda: kda.glu_workspace_size(m(4, 64), m(wrap + 1, 64), m(wrap + 1, 64)))):
        with pytest.raises(ValueError, match=name + ".*32 bits"):
            fn()
