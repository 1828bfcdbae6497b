"""float32 inputs at the ends of their range, on the GPU: the largest and lowest numbers (as masks use them) where the
definition multiplies them by zero or takes them into range, and numbers whose parts in bf16 are subnormal."""
import pytest
import torch

import kda_recurrent_state_amd as kda
from tests import mixer_bounds as MB
from tests import mixer_ref as M
from tests.block_ref import U, bounds_of
from tests.parity import log
from tests.test_gpu_ssm import DEV, F4, call, cpu8, cud, dev, grad, make

pytestmark = pytest.mark.gpu
MOST = torch.finfo(F4).max


def products(T, D=100, F=70, seed=51):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    return r(T, D), r(F, D) * D ** -0.5, r(F, D) * D ** -0.5, 1e-3 * r(T, F)


@pytest.mark.parametrize("act", ["silu", "sigmoid", "gelu"])
@pytest.mark.parametrize("T", [20, 100])
def test_products_of_the_largest_numbers(T, act):
    """In columns where the other factor is zero, and where it is 2^-122."""
    log(f"glu, largest numbers {T} {act}")
    x, wg, wu, dh = products(T)
    x[:, 7], wg[:, 7], wu[:, 7] = 0, 0, 0
    x[:, 8], wg[:, 8], wu[:, 8] = 0, 0, 0
    x[:, 9], wg[:, 9], wu[:, 9] = 0, 0, 2.0 ** -122
    plain = [t.clone() for t in (x, wg, wu)]
    x[3, 7], x[5, 7], x[T - 1, 7] = MOST, -MOST, MOST
    wg[2, 8], wu[4, 8], wg[69, 8] = MOST, -MOST, -MOST
    h = kda.glu_fwd(x.to(DEV), wg.to(DEV), wu.to(DEV), activation=act)
    assert torch.equal(h, kda.glu_fwd(*(t.to(DEV) for t in plain), activation=act))
    x[2, 9], x[6, 9] = 3.4e38, -MOST
    val, bnd = M.glu(x.double(), wg.double(), wu.double(), act, dh.double(), F4)
    args = [t.to(DEV) for t in (x, wg, wu)]
    h, saved = kda.glu_fwd_saved(*args, activation=act)
    M.check(h, val["h"], bnd["h"], "h")
    for got in (kda.glu_bwd(*args, dh.to(DEV), activation=act), kda.glu_bwd(*args, dh.to(DEV), activation=act, saved=saved)):
        for k in got:
            M.check(got[k], val[k], bnd[k], k)


@pytest.mark.parametrize("T", [20, 100])
@pytest.mark.parametrize("scale", [2.0 ** -100, 2.0 ** -118, 2.0 ** -126, 2.0 ** -140])
def test_products_of_small_numbers(T, scale):
    """A factor is held to 2^-134 (half of the least bf16), beside the rounding of products and sums."""
    log(f"glu, small numbers {T} {scale}")
    x, wg, wu, _ = products(T)
    wg.zero_()
    x = x * scale
    u = x.double() @ wu.double().t()
    h, saved = kda.glu_fwd_saved(x.to(DEV), wg.to(DEV), wu.to(DEV), activation="sigmoid")
    off = (6 * x.shape[1] + 16) * U * (x.double().abs() @ wu.double().abs().t()) + 2.0 ** -134 * wu.double().abs().sum(1)
    # a sum below the normal numbers is rounded to 2^-149 each of its 6 D times
    off = off + 6 * x.shape[1] * 2.0 ** -150
    assert ((saved[1].cpu().double() - u).abs() <= off).all() and not saved[0].any()
    assert ((h.cpu().double() - u / 2).abs() <= off + U * u.abs() + 2.0 ** -150).all()


@pytest.mark.parametrize("lengths", [[5], [70, 3], [300]], ids=str)
def test_scan_of_the_largest_numbers(lengths):
    """x where B is zero, and B where x is zero."""
    log(f"ssm, largest numbers {lengths}")
    size = (4, 2, 16, 24)
    v, dy, dhT = make(lengths, size, F4, 52)
    dy, dhT, v["C"], v["D"] = dy * 1e-6, dhT * 1e-6, v["C"] * 1e-3, torch.zeros(4)
    T = sum(lengths)
    at_x, at_b = list(range(0, T, 7)), list(range(3, T, 7))
    v["B"][at_x], v["x"][at_x] = 0, 0
    v["x"][at_b], v["B"][at_b] = 0, 0
    cu, dyd, dhd = cud(lengths), dy.to(DEV), dhT.to(DEV)
    y, h = call(dev(v), cu)
    g = grad(dev(v), dyd, cu, dhd)
    v["x"][at_x, :, 5], v["x"][at_x[::2], 1, 20] = MOST, -MOST
    v["B"][at_b, :, 9], v["B"][at_b[::2], 1, 2] = -MOST, MOST
    y2, h2 = call(dev(v), cu)
    g2 = grad(dev(v), dyd, cu, dhd)
    assert torch.equal(y, y2) and torch.equal(h, h2)
    rest_x = [t for t in range(T) if t not in at_x]
    rest_b = [t for t in range(T) if t not in at_b]
    for k in ("ddt", "dA", "dC", "dh0", "ddt_bias"):
        assert torch.equal(g[k], g2[k]), k
    assert torch.equal(g["dB"][rest_x], g2["dB"][rest_x]) and torch.equal(g["dx"][rest_b], g2["dx"][rest_b])
    val, bnd = MB.grad_bounds(*cpu8(v), bounds_of(lengths), dy.double(), dhT.double())
    for k in val:
        M.check(g2[k], val[k], bnd[k], k)


def test_a_state_of_the_largest_numbers():
    """Read by zeros, and forgotten to where it is in range."""
    log("ssm, states of the largest numbers")
    lengths, size = [40, 3], (4, 2, 16, 24)
    v, _, _ = make(lengths, size, F4, 53)
    v["C"][..., 3] = 0
    v["h0"][:, :, 3, ::2] = MOST
    v["h0"][:, :, 3, 1] = -3.395e38
    val, bnd = M.ssm_bounds(*cpu8(v), bounds_of(lengths))
    y, h = call(dev(v), cud(lengths))
    M.check(y, val["y"], bnd["y"], "y"), M.check(h, val["h"], bnd["h"], "h_T")
    w = dict(v, **{k: v[k][:2] for k in ("x", "dt", "B", "C")})
    val, bnd = M.ssm_bounds(*cpu8(w), [0, 1, 2])
    hs = w["h0"].to(DEV)
    d = dev(w)
    ys, _ = kda.ssm_step(d["x"], d["dt"], d["A"], d["B"], d["C"], hs, d["D"], d["dt_bias"])
    M.check(ys, val["y"], bnd["y"], "y"), M.check(hs, val["h"], bnd["h"], "h")
