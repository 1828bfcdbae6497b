"""The gated products' gradient where offsets pass 32 bits, in whole numbers: sums below 2^24 are exact in any order, so
every value of every gradient has to be the one that chunks of tokens give."""
import pytest
import torch

import kda_recurrent_state_amd as kda
from tests import mixer_ref as M
from tests.parity import log

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F4, BF = torch.float32, torch.bfloat16


# planes of dg and du past 2^32 bytes (bf16, and three of them in fp32), x and dx past 2^32 bytes
@pytest.mark.parametrize("T,D,F,dtype", [(300001, 64, 8192, BF), (100003, 60, 8200, F4), (600001, 4096, 64, BF)], ids=str)
def test_gradient_of_more_than_32_bits(T, D, F, dtype):
    log(f"glu gradient 2^32 bytes {T} {D} {F} {dtype}")
    size = 2 if dtype == BF else 4
    assert max(T * F * size, T * D * size) > 1 << 32 or 3 * 2 * T * F > 1 << 32
    g = torch.Generator(device=DEV).manual_seed(71)
    i = lambda lo, hi, *s: torch.randint(lo, hi + 1, s, generator=g, device=DEV, dtype=torch.int8)
    x, wg, wu = i(-2, 2, T, D).to(dtype), i(-1, 1, F, D).to(dtype), i(-1, 1, F, D).to(dtype)
    # with g = 0 the logistic gate is 1/2 and its slope 1/4: dg = dh u / 4 and du = dh / 2 are whole numbers
    saved = torch.zeros(2, T, F, device=DEV)
    saved[1] = i(-3, 3, T, F)
    dh = i(-1, 1, T, F).to(dtype).mul_(4)
    got = kda.glu_bwd(x, wg, wu, dh, activation="sigmoid", saved=saved)
    dwg, dwu = torch.zeros(F, D, device=DEV), torch.zeros(F, D, device=DEV)
    for a in range(0, T, 20000):
        t = slice(a, min(a + 20000, T))
        d = dh[t].float()
        dg, du, xf = d * saved[1, t] / 4, d / 2, x[t].float()
        assert torch.equal(got["dx"][t], (dg @ wg.float() + du @ wu.float()).to(dtype)), a
        dwg += dg.t().contiguous() @ xf
        dwu += du.t().contiguous() @ xf
    assert max(float(dwg.abs().max()), float(dwu.abs().max())) < 2 ** 24
    assert torch.equal(got["dw_gate"], dwg.to(dtype)) and torch.equal(got["dw_up"], dwu.to(dtype))


def test_gradient_from_the_inputs_alone():
    """Both products computed again, over more than 2^32 bytes: rows at both ends and around the 2^32nd byte."""
    T, D, F = 300001, 64, 8192
    log("glu gradient 2^32 bytes, without kept products")
    g = torch.Generator(device=DEV).manual_seed(72)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV).to(BF)
    x, wg, wu = r(T, D), r(F, D) / 8, r(F, D) / 8
    dh = torch.randn(T, F, generator=g, device=DEV, dtype=BF)
    got = kda.glu_bwd(x, wg, wu, dh, activation="silu")
    edge = (1 << 32) // (2 * F)
    c8 = lambda t: t.cpu().double()
    for a in (0, edge - 5, T - 10):
        t = slice(a, a + 10)
        val, bnd = M.glu(c8(x[t]), c8(wg), c8(wu), "silu", c8(dh[t]), BF)
        M.check(got["dx"][t], val["dx"], bnd["dx"], f"dx from {a}")
    assert torch.isfinite(got["dw_gate"]).all() and torch.isfinite(got["dw_up"]).all()
