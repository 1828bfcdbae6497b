"""Outputs and workspaces that overlap other tensors of a call, refused by the
binding (CPU: the device check and the launch are taken out)."""
import pytest
import torch

import kda_recurrent_state_amd as kda
from kda_recurrent_state_amd import block

T, C, N, W = 200, 8, 2, 4


@pytest.fixture()
def launched(monkeypatch):
    calls = []
    monkeypatch.setattr(block, "_same_device", lambda *a, **k: None)
    monkeypatch.setattr(block, "_launch", lambda fn, lib, device, args: calls.append(fn.__name__))
    return calls


def f(*shape):
    return torch.zeros(*shape)


def within(t, dtype, *shape):
    """A tensor of this type and shape in t's memory, from its first byte."""
    n = torch.empty(shape, dtype=dtype).nbytes
    big = torch.zeros(t.nbytes + n, dtype=torch.uint8)
    return big[:n].view(dtype).view(shape), big[:t.nbytes].view(t.dtype).view(t.shape)


def cu():
    return torch.tensor([0, 50, T], dtype=torch.int32)


# entry point, the names of its tensors in order with a maker of each, keyword ones, and (output: shape and type)
X, LA, ST = (lambda: f(T, C)), (lambda: f(T, C)), (lambda: f(N, C))
STEP, CST = (lambda: f(N, C)), (lambda: f(N, W - 1, C))
WT, B, X3, D1 = (lambda: f(C, W)), (lambda: f(C)), (lambda: f(T, 1, C)), (lambda: f(C))
F32, U8 = torch.float32, torch.uint8
CASES = [
    ("scan_fwd", dict(x=X, log_a=LA, h0=ST, cu_seqlens=cu), dict(out=(F32, T, C), final_state=(F32, N, C))),
    ("scan_fwd_states", dict(x=X, log_a=LA, h0=ST, cu_seqlens=cu),
     dict(out=(F32, T, C), final_state=(F32, N, C), states=(F32, 4, C))),
    ("scan_step", dict(x=STEP, log_a=STEP, h=ST), dict(out=(F32, N, C), h_out=(F32, N, C))),
    ("conv_fwd", dict(x=X, weight=WT, bias=B, state=CST, cu_seqlens=cu),
     dict(out=(F32, T, C), final_state=(F32, N, W - 1, C))),
    ("conv_step", dict(x=STEP, weight=WT, state=CST, bias=B), dict(out=(F32, N, C), state_out=(F32, N, W - 1, C))),
    ("norm_gate_fwd", dict(x=X3, weight=D1, gate=X3), dict(out=(F32, T, 1, C))),
    ("residual_norm_fwd", dict(x=X, residual=X, weight=D1, channel_scale=D1),
     dict(out=(F32, T, C), residual_out=(F32, T, C))),
]
MAY = {("scan_step", "h_out", "h"), ("conv_step", "state_out", "state"), ("norm_gate_fwd", "out", "x"),
       ("residual_norm_fwd", "residual_out", "residual")}  # in place
PAIRS = [(fn, o, i) for fn, ins, outs in CASES for o in outs for i in ins if (fn, o, i) not in MAY]


@pytest.mark.parametrize("fn,out,inp", PAIRS)
def test_an_output_over_an_input(launched, fn, out, inp):
    ins, outs = next((a, b) for g, a, b in CASES if g == fn)
    args = {k: make() for k, make in ins.items()}
    given = {k: torch.zeros(v[1:], dtype=v[0]) for k, v in outs.items()}
    getattr(kda, fn)(**args, **given)  # apart: accepted
    assert len(launched) == 1
    given[out], args[inp] = within(args[inp], *outs[out])
    if inp == "cu_seqlens":
        args[inp].copy_(cu())
    with pytest.raises(ValueError, match="overlaps"):
        getattr(kda, fn)(**args, **given)
    assert len(launched) == 1


WORKSPACE = [
    ("scan_fwd_states", dict(x=X, log_a=LA, h0=ST, cu_seqlens=cu, out=X, final_state=ST, states=lambda: f(4, C))),
    ("scan_bwd", dict(x=X, log_a=LA, dy=X, h0=ST, cu_seqlens=cu, dh_T=ST, states=lambda: f(4, C))),
    ("conv_bwd", dict(x=X, weight=WT, dy=X, bias=B, state=CST, cu_seqlens=cu, dstate_T=CST)),
    ("norm_gate_bwd", dict(x=X3, weight=D1, dy=X3, gate=X3)),
    ("residual_norm_bwd", dict(x=X, residual_out=X, weight=D1, dy=X, dresidual_out=X, channel_scale=D1)),
]


@pytest.mark.parametrize("fn,name", [(fn, n) for fn, a in WORKSPACE for n in a])
def test_a_workspace_over_a_tensor(launched, fn, name):
    args = {k: make() for k, make in next(a for g, a in WORKSPACE if g == fn).items()}
    nbytes = 1 << 20
    getattr(kda, fn)(**args, workspace=torch.zeros(nbytes, dtype=U8))
    assert len(launched) == 1
    ws, args[name] = within(args[name], U8, nbytes)
    if name == "cu_seqlens":
        args[name].copy_(cu())
    with pytest.raises(ValueError, match="overlaps"):
        getattr(kda, fn)(**args, workspace=ws)
    assert len(launched) == 1


def test_a_workspace_is_the_bytes_that_are_needed(launched):
    """What lies behind them in the tensor given as workspace is not the call's."""
    x, la = f(T, C), f(T, C)
    need = kda.scan_workspace_size(x)
    pool = torch.zeros(need + x.nbytes, dtype=U8)
    kda.scan_fwd(pool[need:].view(F32).view(T, C), la, workspace=pool)
    assert launched == ["kda_scan_fwd"]
    with pytest.raises(ValueError, match="overlaps"):
        kda.scan_fwd(pool[need - 4:-4].view(F32).view(T, C), la, workspace=pool)


def rows(buf, every, count):
    return buf[::every][:count]


def test_an_output_between_an_inputs_tokens(launched):
    """Tokens far apart leave room for other tensors: only their own bytes count."""
    buf = f(9, C)
    x, out, la = rows(buf, 4, 2), buf[1:3], f(2, C)  # tokens 0 and 4; rows 1 and 2
    kda.scan_fwd(x, la, out=out)
    kda.scan_step(x, la, f(2, C), out=buf[2:4])
    kda.norm_gate_fwd(x.view(2, 1, C), f(C), out=buf[5:7].view(2, 1, C))
    kda.residual_norm_fwd(la, x, f(C), out=buf[1:3], residual_out=buf[5:7])
    assert len(launched) == 4
    for at in (0, 3, 4):
        with pytest.raises(ValueError, match="overlaps"):
            kda.scan_fwd(x, la, out=buf[at:at + 2])
    flat = buf.view(-1)
    for at in (1, C - 1, 3 * C - C + 1, 5 * C - 1):  # by an element, at either end of either token
        with pytest.raises(ValueError, match="overlaps"):
            kda.scan_fwd(x, la, out=flat[at:at + 2 * C].view(2, C))
    kda.scan_fwd(x, la, out=flat[C:3 * C].view(2, C))
    kda.scan_fwd(x, la, out=flat[2 * C:4 * C].view(2, C))
    kda.scan_fwd(x, la, out=flat[5 * C:7 * C].view(2, C))
    assert len(launched) == 7
    # a slice of a fused projection: every gap is shorter than the output, wherever it lies
    wide = f(T, 3 * C)
    for at in range(0, wide.numel() - T * C + 1, 37):
        with pytest.raises(ValueError, match="overlaps"):
            kda.scan_fwd(wide[:, C:2 * C], f(T, C), out=wide.view(-1)[at:at + T * C].view(T, C))
    assert len(launched) == 7


@pytest.mark.parametrize("seed", range(4))
def test_touching_is_sharing_a_byte(seed):
    """Against the bytes themselves, for token tensors of two and three dimensions."""
    g = torch.Generator().manual_seed(seed)
    pick = lambda lo, hi: int(torch.randint(lo, hi, (1,), generator=g))
    buf = torch.zeros(600)
    base = buf.data_ptr()
    for _ in range(2000):
        n, h, c = pick(0, 5), pick(1, 3), pick(1, 6)
        step, at = pick(h * c, h * c + 40), pick(0, 40)
        t = torch.as_strided(buf, (n, h, c), (step, c, 1), at)
        t = t if pick(0, 2) else torch.as_strided(buf, (n, h * c), (step, 1), at)
        mine = {at + r * step + i for r in range(n) for i in range(h * c)}
        a = pick(0, 300)
        b = a + pick(0, 30)
        assert block._touches(t, base + 4 * a, base + 4 * b) == bool(mine & set(range(a, b)))
