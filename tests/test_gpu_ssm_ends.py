"""The state space scan at the ends of its inputs' range, on the GPU: parameters that are no numbers."""
import pytest
import torch

import kda_recurrent_state_amd as kda
from tests import mixer_ref as M
from tests.parity import log
from tests.test_gpu_ssm import BF, DEV, F4, call, cpu8, cud, dev, grad, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F4, BF])
@pytest.mark.parametrize("name", ["A", "dt_bias"])
@pytest.mark.parametrize("lengths", [[5], [70, 0, 200], [900]], ids=str)
def test_a_nan_parameter_is_its_heads(lengths, name, dtype):
    """As in single steps, every result of that head is NaN, and no other head's bits change."""
    log(f"ssm, a NaN in {name} {lengths} {dtype}")
    v, dy, dhT = make(lengths, (4, 2, 16, 24), dtype, 31)
    d, cu, dyd, dhd = dev(v), cud(lengths), dy.to(DEV), dhT.to(DEV)
    y, h = call(d, cu)
    g = grad(d, dyd, cu, dhd)
    bad = dict(d, **{name: d[name].clone()})
    bad[name][2] = float("nan")
    y2, h2 = call(bad, cu)
    g2 = grad(bad, dyd, cu, dhd)
    keep, full = [0, 1, 3], [n for n, L in enumerate(lengths) if L]
    assert torch.equal(y[:, keep], y2[:, keep]) and torch.equal(h[:, keep], h2[:, keep])
    assert torch.isnan(y2[:, 2]).all() and torch.isnan(h2[full][:, 2]).all()
    for k in ("dx", "ddt", "dh0"):
        assert torch.equal(g[k][:, keep], g2[k][:, keep]), k
    for k in ("dA", "dD", "ddt_bias"):
        assert torch.equal(g[k][keep], g2[k][keep]), k
    assert torch.isnan(g2["dx"][:, 2]).all() and torch.isnan(g2["ddt"][:, 2]).all() and torch.isnan(g2["dA"][2])
    for k in ("dB", "dC"):
        assert torch.equal(g[k][:, 0], g2[k][:, 0]) and torch.isnan(g2[k][:, 1]).all(), k
    if lengths == [5]:
        hs = d["h0"].clone()
        ys, _ = kda.ssm_step(bad["x"][:1], bad["dt"][:1], bad["A"], bad["B"][:1], bad["C"][:1], hs, bad["D"], bad["dt_bias"])
        assert torch.isnan(ys[:, 2]).all() and torch.isnan(hs[:, 2]).all()
        assert torch.isfinite(ys[:, keep]).all() and torch.isfinite(hs[:, keep]).all()


def steep(H=512, T=96, seed=32):
    """Decays of 2^-100 and less: sums of log decays in the thousands, whose differences are what the weights are made
    of.  A token's result is its own weight C d, just above the middle between two bf16 numbers, plus a part of x that puts
    a weight rounded down just below such a middle again: an exponent off by 2^-11 costs a whole step twice."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.rand(*s, generator=g)
    C = (1 + r(T, 1, 1)).to(BF)
    d = (1 + 2.0 ** -8 + 2e-4 + 2e-4 * r(T, H)) / C.float()[:, 0]
    return dict(x=torch.ones(T, H, 1, dtype=BF), dt=d, A=-(140 + 60 * r(H)), B=torch.ones(T, 1, 1, dtype=BF), C=C,
                D=torch.full((H,), 2.0 ** -8 - 2.0 ** -16), dt_bias=torch.zeros(H), h0=torch.zeros(1, H, 1, 1))


def test_weights_behind_steep_decays():
    log("ssm, weights behind steep decays")
    v = steep()
    val, bnd = M.ssm_bounds(*cpu8(v), [0, 96], soft=False, dtype=BF)
    y, h = call(dev(v), softplus=False)
    M.check(y, val["y"], bnd["y"], "y"), M.check(h, val["h"], bnd["h"], "h_T")
    # mild tokens behind steep ones, which see each other
    mild = torch.arange(96) % 32 >= 20
    v["dt"][mild] *= 2.0 ** -9
    val, bnd = M.ssm_bounds(*cpu8(v), [0, 96], soft=False, dtype=BF)
    y, h = call(dev(v), softplus=False)
    M.check(y, val["y"], bnd["y"], "y"), M.check(h, val["h"], bnd["h"], "h_T")
