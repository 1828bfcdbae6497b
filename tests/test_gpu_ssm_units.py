"""The state space scan's gradient where one workgroup takes several of a group's units (a head's blocks of columns),
and over segments: against its float64 definition (tests/mixer_ref.py, tests/mixer_bounds.py)."""
import pytest
import torch

import kda_recurrent_state_amd as kda
from tests import mixer_bounds as MB
from tests import mixer_ref as M
from tests.block_ref import HALF, U, bounds_of
from tests.parity import log
from tests.test_gpu_ssm import BF, DEV, F4, call, cpu8, cud, dev, grad, make

pytestmark = pytest.mark.gpu


def short(n):
    """n sequences of one to three tokens, two of them empty."""
    return [0 if i in (n // 3, n - 1) else 1 + i % 3 for i in range(n)]


# lengths; heads, groups, state, width; units of a group and the workgroups they are shared by in bf16 (a chunk of 64
# tokens) as the plan has it: enough sequences that there are few workgroups to a chunk
CASES = {
    "six units in one": (short(600), (6, 1, 16, 16), 6, 1),
    "ten units in three": (short(200), (10, 1, 33, 40), 10, 3),
    "two blocks a head, four in two": (short(260), (2, 1, 128, 128), 4, 2),
    "two groups, four in one": (short(280), (8, 2, 24, 20), 4, 1),
    "narrow blocks, six in two": (short(300), (2, 1, 200, 70), 6, 2),
    "whole chunks, four in two": ([130] * 10, (64, 16, 16, 16), 4, 2),
    "blocks with an odd end, nine in two": (short(290), (3, 1, 40, 150), 9, 2),
}


@pytest.mark.parametrize("dtype", [F4, BF])
@pytest.mark.parametrize("case", CASES)
def test_units_of_a_workgroup(case, dtype):
    lengths, size, units, shares = CASES[case]
    log(f"ssm gradient, {case} {dtype}")
    H, G, K, P = size
    assert units == H // G * -(-P // (64 if K <= 128 else 32))
    slots = sum(lengths) // 64 + len(lengths)
    assert shares == min(-(-512 // (slots * G)), units) < units
    v, dy, dhT = make(lengths, size, dtype, 21)
    val, bnd = MB.grad_bounds(*cpu8(v), bounds_of(lengths), dy.double(), dhT.double(), dtype=dtype)
    got = grad(dev(v), dy.to(DEV), cud(lengths), dhT.to(DEV))
    w = {k: M.check(got[k], val[k], bnd[k], k) for k in val}
    log("  share of the allowed error: " + " ".join(f"{k} {x:.3f}" for k, x in w.items()))


@pytest.mark.parametrize("dtype", [F4, BF])
@pytest.mark.parametrize("size", [(4, 1, 128, 64), (6, 2, 7, 5), (2, 1, 200, 36)], ids=str)
def test_gradients_that_pass_through_decays(size, dtype):
    """ddt, dA and ddt_bias within the closer bounds."""
    lengths = [130, 3, 201, 0, 60]
    log(f"ssm gradient, closer bounds {size} {dtype}")
    v, dy, dhT = make(lengths, size, dtype, 22)
    val, bnd = MB.grad_bounds(*cpu8(v), bounds_of(lengths), dy.double(), dhT.double(), dtype=dtype)
    got = grad(dev(v), dy.to(DEV), cud(lengths), dhT.to(DEV))
    for k in ("ddt", "dA", "ddt_bias"):
        M.check(got[k], val[k], bnd[k], k)


@pytest.mark.parametrize("dtype", [F4, BF])
def test_segments_against_the_definition(dtype):
    """Sequences of many segments each (of 128 tokens)."""
    lengths, size = [1500, 300], (2, 1, 16, 16)
    log(f"ssm, segments {dtype}")
    v, dy, dhT = make(lengths, size, dtype, 23)
    val, bnd = M.ssm_bounds(*cpu8(v), bounds_of(lengths), dtype=dtype)
    y, h = call(dev(v), cud(lengths))
    M.check(y, val["y"], bnd["y"], "y"), M.check(h, val["h"], bnd["h"], "h_T")
    val, bnd = MB.grad_bounds(*cpu8(v), bounds_of(lengths), dy.double(), dhT.double(), dtype=dtype)
    got = grad(dev(v), dy.to(DEV), cud(lengths), dhT.to(DEV))
    for k in val:
        M.check(got[k], val[k], bnd[k], k)


@pytest.mark.parametrize("dtype", [F4, BF])
def test_segments_against_pieces_by_hand(dtype):
    """Every gradient of a long sequence is that of its pieces, states and derivatives carried from call to call.
    Both are within their bounds of the exact one: R u of the terms' magnitudes, which are the gradients of the absolute
    values (ddt's from its two parts, which have opposite signs there), and 16 u of those with half the decay."""
    T, piece, (H, G, K, P) = 8000, 500, (2, 1, 16, 16)
    log(f"ssm gradient, pieces by hand {dtype}")
    v, dy, dhT = make([T], (H, G, K, P), dtype, 24)
    d, dyd, dhd = dev(v), dy.to(DEV), dhT.to(DEV)
    cut = lambda w, a, h: dict(w, **{k: w[k][a:a + piece] for k in ("x", "dt", "B", "C")}, h0=h)
    got = grad(d, dyd, None, dhd)
    starts = [d["h0"]]
    for a in range(0, T, piece):
        starts.append(call(cut(d, a, starts[-1]))[1])
    g, parts = dhd, []
    for i, a in reversed(list(enumerate(range(0, T, piece)))):
        parts.insert(0, grad(cut(d, a, starts[i]), dyd[a:a + piece], None, g))
        g = parts[0]["dh0"]
    want = {k: torch.cat([p[k] for p in parts]).double() for k in ("dx", "ddt", "dB", "dC")}
    want.update({k: sum(p[k].double() for p in parts) for k in ("dA", "dD", "ddt_bias")}, dh0=g.double())

    def mags(scale):
        m = {k: t.float().abs() if k not in ("dt", "A", "dt_bias") else t for k, t in d.items()}
        m["A"] = d["A"] * scale
        out = {k: t.double() for k, t in grad(m, dyd.float().abs(), None, dhd.abs()).items()}
        z = (m["dt"] + m["dt_bias"]).double()
        step, slope = M.softplus(z), torch.sigmoid(z)
        dxd = (out["dx"] - m["D"].double()[:, None] * dyd.double().abs()) / step[..., None]
        # out = slope (dd + dl A scale), A < 0
        out["ddt"] = slope * 2 * (dxd * m["x"].double()).sum(-1) - out["ddt"]
        out["ddt_bias"] = out["ddt"].sum(0)
        return out

    full, half = mags(1.0), mags(0.5)
    R = 224 + 8 * (6 * K + 6 * P + 64 + H) + 12 * T
    for k in want:
        each = R * full[k] + 16 * half[k]
        if dtype == BF and k in ("dx", "dB", "dC"):
            each = each + (M.BF_OPERAND if k == "dx" else 64) * full[k]
        allowed = 2 * (HALF[got[k].dtype] * (want[k].abs() + each * U) + each * U) + 1e-40
        assert torch.isfinite(got[k]).all(), k
        worst = float(((got[k].double() - want[k]).abs() / allowed).max())
        assert worst <= 1, (k, worst)


@pytest.mark.parametrize("dtype", [F4, BF])
def test_sums_over_many_tokens_keep_their_digits(dtype):
    """dA and ddt_bias of a long sequence, relative to their norms over the heads, within 16 u.

    A token's share of them is off by up to about 24 u in its factors (a step 8 u, four exponentials 4 u each) and by a
    rounding an addition, all of either sign: of 8192 tokens' the sum keeps 24 u / sqrt(8192) times a few.  What does not
    average out is what is off to one side: a tenth of a unit in the last place in every addition of a matrix
    instruction, gathered over the hundreds of additions of a state's memory, was 33 u before the walk's state
    had alternate signs, and terms that cancelled left as much."""
    T, H, K, P = 8192, 4, 64, 64
    log(f"ssm gradient, long sums {dtype}")
    v, dy, dhT = make([T], (H, 1, K, P), dtype, 25)
    d, dyd, dhd = dev(v), dy.to(DEV), dhT.to(DEV)
    got = grad(d, dyd, None, dhd)
    x, dt, A, B, C, bias, h = (d[k].double() for k in ("x", "dt", "A", "B", "C", "dt_bias", "h0"))
    z = dt + bias
    step, slope = M.softplus(z), torch.sigmoid(z)
    a = torch.exp(step * A)
    h, g, before = h[0], dhd[0].double(), torch.empty(T, H, K, P, dtype=torch.float64, device=DEV)
    for t in range(T):
        before[t] = a[t][:, None, None] * h
        h = before[t] + (step[t][:, None] * B[t])[:, :, None] * x[t][:, None]
    dl, dd = torch.empty(T, H, dtype=torch.float64, device=DEV), torch.empty(T, H, dtype=torch.float64, device=DEV)
    dy8 = dyd.double()
    for t in reversed(range(T)):
        g = g + C[t][:, :, None] * dy8[t][:, None]
        dl[t] = (g * before[t]).sum((1, 2))
        dd[t] = ((g * B[t][:, :, None]).sum(1) * x[t]).sum(-1)
        g = a[t][:, None, None] * g
    want = {"dA": (dl * step).sum(0), "ddt_bias": ((dl * A + dd) * slope).sum(0)}
    for k, w in want.items():
        off = float((got[k].double() - w).norm() / w.norm())
        log(f"  {k} {off / U:.2f} u")
        assert off <= 16 * U, (k, off)
