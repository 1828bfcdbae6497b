"""The state space scan, the gated products and the state cache at the limits of their sizes, and calls that run at the same
time, on the GPU."""
import threading

import pytest
import torch

import kda_recurrent_state_amd as kda
from tests import mixer_bounds as MB
from tests import mixer_ref as M
from tests.block_ref import U
from tests.parity import log
from tests.test_gpu_ssm import BF, DEV, F4, call, cpu8, cud, dev, grad, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F4, BF])
def test_widest_state(dtype):
    """256 x 8192: columns do not meet, so results of a column are those of a call on some of the columns, bit for bit, and
    sums over columns are the sums of such calls'."""
    log(f"ssm, widest state {dtype}")
    lengths, K, P, part = [70, 0, 1], 256, 8192, 1024
    v, dy, dhT = make(lengths, (1, 1, K, P), dtype, 81)
    d, cu, dyd, dhd = dev(v), cud(lengths), dy.to(DEV), dhT.to(DEV)
    y, h = call(d, cu)
    g = grad(d, dyd, cu, dhd)
    ys, hs = kda.ssm_step(d["x"][:3], d["dt"][:3], d["A"], d["B"][:3], d["C"][:3], d["h0"], d["D"], d["dt_bias"],
                          h_out=torch.empty_like(d["h0"]))
    sums, mags = {k: 0 for k in ("dB", "dC", "ddt", "dA", "dD", "ddt_bias")}, {}
    for a in range(0, P, part):
        c = slice(a, a + part)
        w = dict(d, x=d["x"][..., c], h0=d["h0"][..., c].contiguous())
        y1, h1 = call(w, cu)
        assert torch.equal(y[..., c], y1) and torch.equal(h[..., c], h1)
        g1 = grad(w, dyd[..., c], cu, dhd[..., c].contiguous())
        assert torch.equal(g["dx"][..., c], g1["dx"]) and torch.equal(g["dh0"][..., c], g1["dh0"])
        for k in sums:
            sums[k] = sums[k] + g1[k].double()
            mags[k] = mags.get(k, 0) + g1[k].double().abs()
        ys1, hs1 = kda.ssm_step(w["x"][:3], w["dt"][:3], w["A"], w["B"][:3], w["C"][:3], w["h0"], w["D"], w["dt_bias"],
                                h_out=torch.empty_like(w["h0"]))
        assert torch.equal(hs[..., c], hs1)
        # a step's sum over the rows is shared by fewer or more lanes: y in another order
        assert ((ys[..., c] - ys1).abs() <= (ys1.abs() * (2 ** -7 if dtype == BF else 2 ** -23) + 512 * U * ys1.abs().amax())).all()
    for k in sums:
        # each part is off by its own rounding (half a step of its type); the sums' own, of 8 parts and of 6 K + 6 P products
        # a term, are far below what a lost part would be: 2^-10 of the parts' magnitudes
        off = (g[k].double() - sums[k]).abs()
        assert (off <= 2.0 ** -7 * mags[k] if g[k].dtype == BF else off <= 2.0 ** -10 * (mags[k] + mags[k].amax())).all(), k


@pytest.mark.parametrize("dtype", [F4, BF])
@pytest.mark.parametrize("G", [1, 65536])
def test_most_heads(G, dtype):
    log(f"ssm, 65536 heads in {G} groups {dtype}")
    lengths, size = [2, 0, 1], (65536, G, 1, 1)
    v, dy, dhT = make(lengths, size, dtype, 82)
    val, bnd = M.ssm_bounds(*cpu8(v), [0, 2, 2, 3], dtype=dtype)
    d, cu = dev(v), cud(lengths)
    y, h = call(d, cu)
    M.check(y, val["y"], bnd["y"], "y"), M.check(h, val["h"], bnd["h"], "h_T")
    val, bnd = MB.grad_bounds(*cpu8(v), [0, 2, 2, 3], dy.double(), dhT.double(), dtype=dtype)
    got = grad(d, dy.to(DEV), cu, dhT.to(DEV))
    for k in val:
        M.check(got[k], val[k], bnd[k], k)


def test_many_sequences():
    """60000 of one token, and every seventh of none: the formula itself."""
    log("ssm, many sequences")
    N, (H, G, K, P) = 60000, (2, 1, 4, 4)
    lengths = [0 if n % 7 == 3 else 1 for n in range(N)]
    T = sum(lengths)
    v, dy, dhT = make([T], (H, G, K, P), F4, 83)
    v["h0"] = 0.3 * torch.randn(N, H, K, P, generator=torch.Generator().manual_seed(84))
    cu = torch.tensor([0] + torch.tensor(lengths).cumsum(0).tolist(), dtype=torch.int32, device=DEV)
    y, h = call(dev(v), cu)
    x, dt, A, B, C, D, bias, h0 = cpu8(v)
    has = torch.tensor(lengths, dtype=torch.bool)
    step = M.softplus(dt + bias)
    state = torch.exp(step * A)[:, :, None, None] * h0[has]
    add = (step[:, :, None] * B)[..., None] * x[:, :, None]
    want = h0.clone()
    want[has] = state + add
    mag = state.abs() + add.abs()
    off = 250 * U * mag  # R of mixer_ref for a token, without the sums over rows
    assert ((h.cpu().double()[has] - want[has]).abs() <= off).all() and torch.equal(h.cpu()[~has], v["h0"][~has])
    yw = (C[:, 0][:, None, :, None] * want[has]).sum(2) + D[:, None] * x
    ym = (C[:, 0][:, None, :, None].abs() * mag).sum(2) + (D[:, None] * x).abs()
    assert ((y.cpu().double() - yw).abs() <= (250 + 8 * (6 * K + 64)) * U * ym).all()
    g = grad(dev(v), dy.to(DEV), cu, None, initial_state_grad=True)
    dh0 = torch.zeros_like(h0)
    dh0[has] = torch.exp(step * A)[:, :, None, None] * C[:, 0][:, None, :, None] * dy.double()[:, :, None]
    assert ((g["dh0"].cpu().double() - dh0).abs() <= 250 * U * dh0.abs()).all()


@pytest.mark.parametrize("dtype", [F4, BF])
@pytest.mark.parametrize("T,D,F", [(3, 1 << 20, 2), (66, 1 << 20, 1), (3, 2, 1 << 20), (66, 1, 1 << 20)], ids=str)
def test_widest_products(T, D, F, dtype):
    log(f"glu, widest {T} {D} {F} {dtype}")
    g = torch.Generator().manual_seed(85)
    r = lambda *s: torch.randn(*s, generator=g)
    x, wg, wu, dh = r(T, D).to(dtype), (r(F, D) * D ** -0.5).to(dtype), (r(F, D) * D ** -0.5).to(dtype), r(T, F).to(dtype)
    val, bnd = M.glu(x.double(), wg.double(), wu.double(), "silu", dh.double(), dtype)
    args = [t.to(DEV) for t in (x, wg, wu)]
    M.check(kda.glu_fwd(*args), val["h"], bnd["h"], "h")
    got = kda.glu_bwd(*args, dh.to(DEV))
    for k in got:
        M.check(got[k], val[k], bnd[k], k)


@pytest.mark.parametrize("fmt", [torch.int8, torch.float8_e4m3fn])
def test_most_states(fmt):
    log(f"state cache, 2^20 states {fmt}")
    R = 1 << 20
    x = torch.randn(R, 2, 3, generator=torch.Generator().manual_seed(86))
    codes, scales = kda.state_cache_empty(R + 5, x.shape[1:], fmt, DEV)
    kda.state_cache_write(x.to(DEV), codes, scales)
    want, ws = M.quantise(x, fmt)
    assert torch.equal(scales[:R].cpu(), ws) and torch.equal(codes[:R].float().cpu().double(), want)
    assert not codes[R:].view(torch.int8).any() and not scales[R:].any()
    out = torch.empty(R, 2, 3, device=DEV)
    kda.state_cache_read(codes[:R], scales[:R], out=out)
    assert torch.equal(out.cpu(), want.float() * ws[..., None])


def test_calls_at_the_same_time():
    """Three threads, a stream each, calls of every operator between each other: results of each are those of a call alone."""
    log("calls of three threads")
    lengths = [300, 5, 0, 130]
    jobs = []
    for n in range(3):
        v, dy, dhT = make(lengths, (4, 2, 32, 40), BF if n != 1 else F4, 90 + n)
        g = torch.Generator().manual_seed(95 + n)
        r = lambda *s: torch.randn(*s, generator=g).to(DEV)
        jobs.append((dev(v), dy.to(DEV), dhT.to(DEV), cud(lengths), r(90, 100), r(70, 100), r(70, 100), r(90, 70), r(5, 4, 32, 40)))

    def work(job):
        d, dy, dhT, cu, x, wg, wu, dh, states = job
        y, h = call(d, cu)
        g = grad(d, dy, cu, dhT)
        codes, scales = kda.state_cache_empty(6, states.shape[1:], torch.float8_e4m3fn, DEV)
        slots = torch.tensor([5, 0, 2, 2, 1], dtype=torch.int32, device=DEV)
        kda.state_cache_write(states, codes, scales, slots)
        f = kda.glu_bwd(x, wg, wu, dh)
        return [y, h, *g.values(), kda.glu_fwd(x, wg, wu), *f.values(), kda.state_cache_read(codes, scales, slots)]

    want = [work(j) for j in jobs]
    torch.cuda.synchronize()
    got, errors = [[] for _ in jobs], []

    def run(n):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(20):
                    got[n].append(work(jobs[n]))
            stream.synchronize()
        except Exception as e:  # reported by the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=run, args=(n,)) for n in range(3)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors, errors
    for n in range(3):
        for one in got[n]:
            assert all(torch.equal(a, b) for a, b in zip(one, want[n]))
