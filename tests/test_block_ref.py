"""The float64 references of the operators around the state layer: their
gradients against central differences of their forwards (CPU)."""
import pytest
import torch

from tests import block_ref as R

F8 = torch.float64


def gen(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, dtype=F8)


def differences(fn, arg, dirs, eps=1e-6):
    """Central differences of the scalar fn along each direction."""
    return [float(fn(arg + eps * v) - fn(arg - eps * v)) / (2 * eps) for v in dirs]


def agree(fn, arg, grad, r, name):
    dirs = [r(*arg.shape) for _ in range(3)]
    for v, d in zip(dirs, differences(fn, arg, dirs)):
        want = float((grad * v).sum())
        # the difference's truncation and rounding: eps^2 and 1e-16 / eps of the values
        assert abs(d - want) <= 1e-6 * (1 + abs(want)), (name, d, want)


LENGTHS = [0, 1, 5, 0, 9, 2, 0]


def test_scan_gradient_against_differences():
    r = gen(1)
    cu, C = R.bounds_of(LENGTHS), 3
    T, N = cu[-1], len(LENGTHS)
    args = dict(x=r(T, C), la=-r(T, C).abs(), h0=r(N, C))
    dy, dhT = r(T, C), r(N, C)

    def loss(**kw):
        v, _ = R.scan(**{**args, **kw}, cu=cu)
        return (v["y"] * dy).sum() + (v["h"] * dhT).sum()

    val, _ = R.scan_grad(**args, cu=cu, dy=dy, dhT=dhT)
    for k, g in (("x", "dx"), ("la", "dlog_a"), ("h0", "dh0")):
        agree(lambda a: loss(**{k: a}), args[k], val[g], r, g)


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("silu", [False, True])
def test_conv_gradient_against_differences(W, silu):
    r = gen(2)
    cu, C = R.bounds_of(LENGTHS), 3
    T, N = cu[-1], len(LENGTHS)
    args = dict(x=r(T, C), w=r(C, W), b=r(C), state=r(N, W - 1, C))
    dy, dsT = r(T, C), r(N, W - 1, C)

    def loss(**kw):
        v, _ = R.conv(**{**args, **kw}, cu=cu, silu=silu)
        return (v["y"] * dy).sum() + (v["state"] * dsT).sum()

    val, _ = R.conv_grad(**args, cu=cu, silu=silu, dy=dy, dsT=dsT)
    for k, g in (("x", "dx"), ("w", "dweight"), ("b", "dbias"), ("state", "dstate")):
        agree(lambda a: loss(**{k: a}), args[k], val[g], r, g)


@pytest.mark.parametrize("act", ["silu", "sigmoid", None])
def test_norm_gate_gradient_against_differences(act):
    r = gen(3)
    args = dict(x=r(4, 2, 7), w=r(7), g=None if act is None else r(4, 2, 7))
    dy = r(4, 2, 7)

    def loss(**kw):
        return (R.norm_gate(**{**args, **kw}, act=act, eps=1e-3)[0] * dy).sum()

    val, _ = R.norm_gate_grad(**args, act=act, eps=1e-3, dy=dy)
    for k, g in (("x", "dx"), ("w", "dweight"), ("g", "dgate")):
        if args[k] is not None:
            agree(lambda a: loss(**{k: a}), args[k], val[g], r, g)


@pytest.mark.parametrize("with_cs", [False, True])
def test_residual_norm_gradient_against_differences(with_cs):
    r = gen(4)
    T, D = 5, 9
    x, res, w, cs = r(T, D), r(T, D), r(D), r(D) if with_cs else None
    dy, dres = r(T, D), r(T, D)

    def loss(x=x, res=res, w=w, cs=cs):
        v, _ = R.residual_norm(x, res, w, 0.5, cs, 1e-3)
        return (v["y"] * dy).sum() + (v["residual"] * dres).sum()

    h = R.residual_norm(x, res, w, 0.5, cs, 1e-3)[0]["residual"]
    val, _ = R.residual_norm_grad(x, h, w, 0.5, cs, 1e-3, dy, dres)
    agree(lambda a: loss(x=a), x, val["dx"], r, "dx")
    agree(lambda a: loss(res=a), res, val["dresidual"], r, "dresidual")
    agree(lambda a: loss(w=a), w, val["dweight"], r, "dweight")
    if with_cs:
        agree(lambda a: loss(cs=a), cs, val["dchannel_scale"], r, "dchannel_scale")
