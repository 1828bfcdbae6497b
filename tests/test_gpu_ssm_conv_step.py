"""One token behind the convolution without an activation and without the optional parameters, on the GPU against the
definition: the results, both states, and what a call with them gives stays apart."""
import pytest
import torch

import kda_recurrent_state_amd as kda
from tests import mixer_ref as M
from tests.parity import log
from tests.test_gpu_ssm import BF, DEV, F4, make, slice_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F4, BF])
@pytest.mark.parametrize("optional", ["none", "all", "conv_bias", "D", "dt_bias"])
@pytest.mark.parametrize("activation", [None, "silu"])
@pytest.mark.parametrize("taps", [2, 3, 4])
@pytest.mark.parametrize("size", [(4, 1, 128, 64), (6, 2, 7, 5)], ids=str)
def test_convolution_and_scan(size, taps, activation, optional, dtype):
    log(f"ssm_conv_step {size} {taps} {activation} {optional} {dtype}")
    H, G, K, P = size
    N, ch = 3, H * P + 2 * G * K
    g = torch.Generator().manual_seed(41)
    r = lambda *s: torch.randn(*s, generator=g)
    xbc, w, b, st = r(N, ch).to(dtype), r(ch, taps) * taps ** -0.5, r(ch) * 0.1, r(N, taps - 1, ch).to(dtype)
    v, _, _ = make([1] * N, size, dtype, 42)
    has = lambda name: optional in ("all", name)
    bias8, D8, dtb8 = (t.double() if has(n) else torch.zeros_like(t).double()
                       for n, t in (("conv_bias", b), ("D", v["D"]), ("dt_bias", v["dt_bias"])))
    full = torch.cat([st, xbc[:, None]], 1).double()
    w8 = w.double().t()
    z = bias8 + (full * w8).sum(1)
    s = z * torch.sigmoid(z) if activation else z
    cut = lambda t: (t[:, :H * P].reshape(N, H, P), t[:, H * P:H * P + G * K].reshape(N, G, K), t[:, H * P + G * K:].reshape(N, G, K))
    x, B, C = cut(s)
    dt, A, h0 = (v[k].double() for k in ("dt", "A", "h0"))
    val, bnd = M.ssm_bounds(x, dt, A, B, C, D8, dtb8, h0, list(range(N + 1)))
    # the convolved values: (taps + 2) roundings of the sum's terms, whose slope SiLU takes 1.1 times at most, and
    # SiLU's own (|z| + 8) u
    sums = (taps + 2) * (bias8.abs() + (full.abs() * w8.abs()).sum(1))
    e = 1.1 * sums + (z.abs() + 8) * s.abs() if activation else sums
    ex, eB, eC = cut(e)
    step = M.softplus(dt + dtb8)
    rep = lambda t: t.abs().repeat_interleave(H // G, 1)
    eh = step[:, :, None, None] * (rep(eB)[..., None] * x.abs()[:, :, None] + rep(B)[..., None] * ex[:, :, None])
    ey = (rep(C)[..., None] * eh + rep(eC)[..., None] * val["h"].abs()).sum(2) + D8.abs()[:, None] * ex
    on = lambda name, t: t.to(DEV) if has(name) else None
    h, cs = v["h0"].to(DEV), st.to(DEV)
    y, cso, ho = kda.ssm_conv_step(xbc.to(DEV), w.to(DEV), cs, v["dt"].to(DEV), v["A"].to(DEV), h, on("D", v["D"]),
                                   on("dt_bias", v["dt_bias"]), on("conv_bias", b), activation=activation)
    assert cso is cs and ho is h
    M.check(y, val["y"], bnd["y"] + 1.01 * ey, "y")
    M.check(h, val["h"], bnd["h"] + 1.01 * eh, "h")
    assert torch.equal(cs.cpu(), full[:, 1:].to(dtype))
    # from a slice, states apart, in a given workspace that holds no numbers
    ws = torch.full((kda.ssm_conv_step_workspace_size(xbc.to(DEV), h),), 255, dtype=torch.uint8, device=DEV)
    h2, cs2, h_in, cs_in = torch.empty_like(h), torch.empty_like(cs), v["h0"].to(DEV), st.to(DEV)
    y2, _, _ = kda.ssm_conv_step(slice_of(xbc.to(DEV)), w.to(DEV), cs_in, v["dt"].to(DEV), v["A"].to(DEV), h_in, on("D", v["D"]),
                                 on("dt_bias", v["dt_bias"]), on("conv_bias", b), activation=activation, h_out=h2,
                                 conv_state_out=cs2, workspace=ws)
    assert torch.equal(y, y2) and torch.equal(h, h2) and torch.equal(cs, cs2)
    assert torch.equal(h_in.cpu(), v["h0"]) and torch.equal(cs_in.cpu(), st)
