"""The selective state space scan on the GPU against its float64 definition (tests/mixer_ref.py, which also
derives the tolerances)."""
import pytest
import torch

import kda_recurrent_state_amd as kda
from tests import mixer_ref as M
from tests.block_ref import bounds_of
from tests.parity import log

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F8, F4, BF = torch.float64, torch.float32, torch.bfloat16
LENS = {"one": [1], "short": [1] * 40, "edges": [0, 1, 0, 31, 64, 63, 65, 0, 33, 0], "long": [300], "pair": [128, 128],
        "ragged": [130, 3, 201, 60]}
# heads, groups, state, width: every compiled state block, whole and odd
SIZES = [(4, 1, 128, 64), (2, 2, 16, 16), (6, 2, 7, 5), (3, 1, 40, 50), (2, 1, 128, 130), (2, 1, 200, 36), (4, 2, 64, 32),
         (10, 2, 33, 66), (1, 1, 1, 1)]


def make(lengths, size, dtype, seed, fast=False):
    H, G, K, P = size
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    T, N = sum(lengths), len(lengths)
    v = dict(x=r(T, H, P).to(dtype), dt=r(T, H), A=-(torch.rand(H, generator=g) * 15 + 1), B=r(T, G, K).to(dtype),
             C=r(T, G, K).to(dtype), D=r(H), dt_bias=r(H) * 0.5 - (0.0 if fast else 4.0), h0=r(N, H, K, P) * 0.3)
    return v, r(T, H, P).to(dtype), r(N, H, K, P) * 0.2


def bounds(v, lengths, **kw):
    return M.ssm_bounds(*cpu8(v), bounds_of(lengths), dtype=v["x"].dtype, **kw)


def grad_bounds(v, lengths, dy, dhT, **kw):
    return M.ssm_grad_bounds(*cpu8(v), bounds_of(lengths), dy.double(), dhT.double(), dtype=v["x"].dtype, **kw)


def cpu8(v):
    return [v[k].double() for k in ("x", "dt", "A", "B", "C", "D", "dt_bias", "h0")]


def dev(v):
    return {k: t.to(DEV) for k, t in v.items()}


def cud(lengths):
    return torch.tensor(bounds_of(lengths), dtype=torch.int32, device=DEV)


def slice_of(t):
    wide = torch.full((t.shape[0], 3) + tuple(t.shape[1:]), 7.0, dtype=t.dtype, device=t.device)
    wide[:, 1] = t
    return wide[:, 1]


def call(v, cu=None, **kw):
    return kda.ssm_fwd(v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], v["dt_bias"], v["h0"], cu, **kw)


def grad(v, dy, cu=None, dhT=None, **kw):
    return kda.ssm_bwd(v["x"], v["dt"], v["A"], v["B"], v["C"], dy, v["D"], v["dt_bias"], v["h0"], cu, dhT, **kw)


@pytest.mark.parametrize("dtype", [F4, BF])
@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("lens", LENS)
def test_forward(lens, size, dtype):
    lengths = LENS[lens]
    log(f"ssm forward {lens} {size} {dtype}")
    v, _, _ = make(lengths, size, dtype, 3)
    val, bnd = bounds(v, lengths)
    d = dev(v)
    y, h = call(d, cud(lengths))
    w = [M.check(y, val["y"], bnd["y"], "y"), M.check(h, val["h"], bnd["h"], "h_T")]
    s = dict(d, **{k: slice_of(d[k]) for k in ("x", "dt", "B", "C")})
    y2, h2 = call(s, cud(lengths))
    assert torch.equal(y, y2) and torch.equal(h, h2)
    log("  share of the allowed error: " + " ".join(f"{x:.3f}" for x in w))


@pytest.mark.parametrize("dtype", [F4, BF])
@pytest.mark.parametrize("size", [s for s in SIZES if s != (2, 1, 128, 130)], ids=str)
@pytest.mark.parametrize("lens", ["one", "edges", "long", "ragged"])
def test_gradient(lens, size, dtype):
    lengths = LENS[lens]
    log(f"ssm gradient {lens} {size} {dtype}")
    v, dy, dhT = make(lengths, size, dtype, 4)
    val, bnd = grad_bounds(v, lengths, dy, dhT)
    d, dyd, dhd = dev(v), dy.to(DEV), dhT.to(DEV)
    got = grad(d, dyd, cud(lengths), dhd)
    w = {k: M.check(got[k], val[k], bnd[k], k) for k in val}
    s = dict(d, **{k: slice_of(d[k]) for k in ("x", "dt", "B", "C")})
    again = grad(s, slice_of(dyd), cud(lengths), dhd)
    assert all(torch.equal(got[k], again[k]) for k in got)
    log("  share of the allowed error: " + " ".join(f"{k} {x:.3f}" for k, x in w.items()))


@pytest.mark.parametrize("dtype", [F4, BF])
def test_any_decay(dtype):
    """Steps that forget everything next to steps that forget nothing, and steps of zero."""
    lengths, size = [200, 70], (4, 1, 32, 32)
    v, dy, dhT = make(lengths, size, dtype, 5, fast=True)
    v["dt_bias"].zero_()
    T = sum(lengths)
    v["dt"] = torch.full((T, 4), 1e-3)
    v["dt"][10:14, 0] = 60.0     # |log decay| far past what fp32 holds
    v["dt"][30:90, 1] = 7.0      # a long steep stretch, then mild tokens
    v["dt"][::3, 2] = 0.0
    v["dt"][100, 3] = 5.0
    val, bnd = bounds(v, lengths, soft=False)
    d, cu = dev(v), cud(lengths)
    y, h = call(d, cu, softplus=False)
    M.check(y, val["y"], bnd["y"], "y"), M.check(h, val["h"], bnd["h"], "h_T")
    val, bnd = grad_bounds(v, lengths, dy, dhT, soft=False)
    got = grad(d, dy.to(DEV), cu, dhT.to(DEV), softplus=False)
    for k in val:
        M.check(got[k], val[k], bnd[k], k)


def test_optional_arguments():
    lengths, size = [70, 20], (4, 2, 16, 24)
    v, dy, dhT = make(lengths, size, F4, 6)
    zero = dict(v, D=torch.zeros(4), dt_bias=torch.zeros(4), h0=torch.zeros_like(v["h0"]))
    val, bnd = bounds(zero, lengths)
    d, cu = dev(dict(v, dt_bias=v["dt_bias"])), cud(lengths)
    none = dict(d, D=None, dt_bias=None, h0=None)
    y, h = call(none, cu)
    M.check(y, val["y"], bnd["y"], "y"), M.check(h, val["h"], bnd["h"], "h_T")
    assert call(none, cu, final_state=False)[1] is None
    gz = dev(zero)
    full, got = grad(gz, dy.to(DEV), cu, torch.zeros_like(gz["h0"])), grad(none, dy.to(DEV), cu, initial_state_grad=False)
    assert got["dD"] is None and got["ddt_bias"] is None and got["dh0"] is None
    for k in ("dx", "ddt", "dA", "dB", "dC"):
        assert torch.equal(full[k], got[k]), k
    # equal lengths without offsets
    v, dy, dhT = make([64, 64, 64], size, BF, 7)
    d = dev(v)
    a, b = call(d, cud([64, 64, 64])), call(d, num_seqs=3)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a, b = grad(d, dy.to(DEV), cud([64, 64, 64]), dhT.to(DEV)), grad(d, dy.to(DEV), None, dhT.to(DEV), num_seqs=3)
    assert all(torch.equal(a[k], b[k]) for k in a)


@pytest.mark.parametrize("dtype", [F4, BF])
def test_rows_behind_the_last_sequence(dtype):
    """They may hold anything, and their rows of the outputs stay."""
    lengths, size = [50, 33], (4, 2, 24, 20)
    v, dy, dhT = make(lengths + [40], size, dtype, 8)
    v["h0"], dhT = v["h0"][:2].contiguous(), dhT[:2].contiguous()
    d, cu, T = dev(v), cud(lengths), 83
    want = call({k: (t[:T] if k in ("x", "dt", "B", "C") else t) for k, t in d.items()}, cu)
    wantg = grad({k: (t[:T] if k in ("x", "dt", "B", "C") else t) for k, t in d.items()}, dy.to(DEV)[:T], cu, dhT.to(DEV))
    for k in ("x", "dt", "B", "C"):
        d[k][T:] = float("nan")
    dyd = dy.to(DEV)
    dyd[T:] = float("inf")
    out = torch.full_like(d["x"], 5.0)
    y, h = call(d, cu, out=out)
    assert torch.equal(y[:T], want[0]) and torch.equal(h, want[1]) and (y[T:] == 5).all()
    got = grad(d, dyd, cu, dhT.to(DEV))
    for k in got:
        assert torch.equal(got[k][:T] if k in ("dx", "ddt", "dB", "dC") else got[k], wantg[k]), k


@pytest.mark.parametrize("dtype", [F4, BF])
def test_a_non_finite_value_stays_in_its_sequence(dtype):
    lengths, size = [40, 150, 40], (4, 1, 32, 40)
    v, dy, dhT = make(lengths, size, dtype, 9)
    d, cu = dev(v), cud(lengths)
    y, h = call(d, cu)
    g = grad(d, dy.to(DEV), cu, dhT.to(DEV))
    d["x"][100, 2, 3] = float("nan")
    d["B"][120, 0, 1] = float("inf")
    y2, h2 = call(d, cu)
    g2 = grad(d, dy.to(DEV), cu, dhT.to(DEV))
    keep = [slice(0, 40), slice(190, 230)]
    for s in keep:
        assert torch.equal(y[s], y2[s])
        for k in ("dx", "ddt", "dB", "dC"):
            assert torch.equal(g[k][s], g2[k][s]), k
    assert torch.equal(h[0], h2[0]) and torch.equal(h[2], h2[2])
    assert torch.equal(y[40:100 - 63], y2[40:100 - 63]) and not torch.isfinite(y2[100:190, 2, 3]).any()


def test_no_tokens_and_no_sequences():
    v, dy, dhT = make([0, 0], (4, 2, 16, 24), BF, 10)
    d = dev(v)
    y, h = call(d, cud([0, 0]))
    assert y.shape[0] == 0 and torch.equal(h, d["h0"])
    got = grad(d, dy.to(DEV), cud([0, 0]), dhT.to(DEV))
    assert torch.equal(got["dh0"], dhT.to(DEV)) and all(not got[k].any() for k in ("dA", "dD", "ddt_bias"))
    e = {k: t[:0] if k in ("h0",) else t for k, t in d.items()}
    y, h = call(e, cud([]))
    assert h.shape[0] == 0
    assert not grad(e, dy.to(DEV), cud([]), dhT.to(DEV)[:0])["dA"].any()


@pytest.mark.parametrize("dtype", [F4, BF])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_step(size, dtype):
    H, G, K, P = size
    N = 5
    v, _, _ = make([1] * N, size, dtype, 11)
    val, bnd = M.ssm_bounds(*cpu8(v), list(range(N + 1)))
    d = dev(v)
    h = d["h0"].clone()
    args = (d["x"], d["dt"], d["A"], d["B"], d["C"])
    y, ho = kda.ssm_step(*args, h, d["D"], d["dt_bias"])
    assert ho is h
    M.check(y, val["y"], bnd["y"], "y"), M.check(h, val["h"], bnd["h"], "h")
    h2 = torch.empty_like(h)
    y2, _ = kda.ssm_step(*(slice_of(t) if i != 2 else t for i, t in enumerate(args)), d["h0"], d["D"], d["dt_bias"], h_out=h2)
    assert torch.equal(y, y2) and torch.equal(h, h2)


@pytest.mark.parametrize("dtype", [F4, BF])
@pytest.mark.parametrize("taps", [2, 3, 4])
@pytest.mark.parametrize("size", [(4, 1, 128, 64), (6, 2, 7, 5), (2, 2, 40, 70)], ids=str)
def test_step_behind_its_convolution(size, taps, dtype):
    """Against the definition: the convolution's own, then the scan's, nothing rounded between."""
    H, G, K, P = size
    N, C = 3, H * P + 2 * G * K
    g = torch.Generator().manual_seed(12)
    r = lambda *s: torch.randn(*s, generator=g)
    xbc, w, b, st = r(N, C).to(dtype), r(C, taps) * taps ** -0.5, r(C) * 0.1, r(N, taps - 1, C).to(dtype)
    v, _, _ = make([1] * N, size, dtype, 13)
    full = torch.cat([st, xbc[:, None]], 1).double()
    z = b.double() + (full * w.double().t()).sum(1)
    s = z * torch.sigmoid(z)
    x, B, Cm = s[:, :H * P].reshape(N, H, P), s[:, H * P:H * P + G * K].reshape(N, G, K), s[:, H * P + G * K:].reshape(N, G, K)
    rest = [v[k].double() for k in ("dt", "A", "D", "dt_bias", "h0")]
    val, bnd = M.ssm_bounds(x, rest[0], rest[1], B, Cm, rest[2], rest[3], rest[4], list(range(N + 1)))
    # the convolved values are off by at most e: (taps + 2) roundings of the sum's terms, and SiLU's (|z| + 6) u
    e = (taps + 2) * (b.double().abs() + (full.abs() * w.double().abs().t()).sum(1)) * 1.1 + (z.abs() + 8) * s.abs()
    ex, eB, eC = e[:, :H * P].reshape(N, H, P), e[:, H * P:H * P + G * K].reshape(N, G, K), e[:, H * P + G * K:].reshape(N, G, K)
    d8 = M.softplus(rest[0] + rest[3])
    per = H // G
    rep = lambda t: t.abs().repeat_interleave(per, 1)
    eh = d8[:, :, None, None] * (rep(eB)[..., None] * x.abs()[:, :, None] + rep(B)[..., None] * ex[:, :, None])
    ey = (rep(Cm)[..., None] * eh + rep(eC)[..., None] * val["h"].abs()).sum(2) + rest[2].abs()[:, None] * ex
    dd = dev(v)
    h, cs = dd["h0"].clone(), st.to(DEV)
    args = (dd["dt"], dd["A"])
    y, cso, ho = kda.ssm_conv_step(xbc.to(DEV), w.to(DEV), cs, *args, h, dd["D"], dd["dt_bias"], b.to(DEV))
    assert cso is cs and ho is h
    M.check(y, val["y"], bnd["y"] + 1.01 * ey, "y")
    M.check(h, val["h"], bnd["h"] + 1.01 * eh, "h")
    assert torch.equal(cs.cpu(), full[:, 1:].to(dtype))
    # apart from its inputs, from a slice, without activation and bias
    cs2, h2 = torch.empty_like(cs), torch.empty_like(h)
    y2, _, _ = kda.ssm_conv_step(slice_of(xbc.to(DEV)), w.to(DEV), st.to(DEV), *args, dd["h0"], dd["D"], dd["dt_bias"],
                                 b.to(DEV), conv_state_out=cs2, h_out=h2)
    assert torch.equal(y, y2) and torch.equal(cs, cs2) and torch.equal(h, h2)
    y3, _, _ = kda.ssm_conv_step(xbc.to(DEV), w.to(DEV), st.to(DEV), *args, dd["h0"].clone(), activation=None)
    assert torch.isfinite(y3).all()


def test_steps_are_the_scan():
    T, size = 70, (4, 2, 64, 64)
    v, _, _ = make([T], size, F4, 14)
    val, bnd = M.ssm_bounds(*cpu8(v), [0, T])
    d = dev(v)
    h = d["h0"].clone()
    for t in range(T):
        s = slice(t, t + 1)
        y, _ = kda.ssm_step(d["x"][s], d["dt"][s], d["A"], d["B"][s], d["C"][s], h, d["D"], d["dt_bias"])
        M.check(y, val["y"][s], bnd["y"][s], f"y of token {t}")
    M.check(h, val["h"], bnd["h"], "h")


def test_states_continue():
    """A sequence in two calls is the sequence in one, to rounding; its gradient as well."""
    lengths, size = [190], (4, 1, 40, 30)
    v, dy, dhT = make(lengths, size, F4, 15)
    d = dev(v)
    val, bnd = M.ssm_bounds(*cpu8(v), [0, 190])
    cut = lambda a, b, h: dict(d, **{k: d[k][a:b] for k in ("x", "dt", "B", "C")}, h0=h)
    y1, h1 = call(cut(0, 77, d["h0"]))
    y2, h2 = call(cut(77, 190, h1))
    M.check(torch.cat([y1, y2]), val["y"], 2 * bnd["y"], "y"), M.check(h2, val["h"], 2 * bnd["h"], "h")
    gval, gb = M.ssm_grad_bounds(*cpu8(v), [0, 190], dy.double(), dhT.double())
    dyd = dy.to(DEV)
    b2 = grad(cut(77, 190, h1), dyd[77:], None, dhT.to(DEV))
    b1 = grad(cut(0, 77, d["h0"]), dyd[:77], None, b2["dh0"])
    for k in ("dx", "ddt", "dB", "dC"):
        M.check(torch.cat([b1[k], b2[k]]), gval[k], 2 * gb[k], k)
    for k in ("dA", "dD", "ddt_bias"):
        M.check(b1[k] + b2[k], gval[k], 2 * gb[k], k)
    M.check(b1["dh0"], gval["dh0"], 2 * gb["dh0"], "dh0")


@pytest.mark.parametrize("dtype", [F4, BF])
def test_long_sequences_in_segments(dtype):
    """Enough tokens for many segments: against the same call with every sequence's state carried by hand."""
    size, T = (2, 1, 16, 16), 40000
    v, dy, dhT = make([T], size, dtype, 16)
    d = dev(v)
    y, h = call(d)
    hh, parts = d["h0"], []
    for a in range(0, T, 1000):
        p, hh = call(dict(d, **{k: d[k][a:a + 1000] for k in ("x", "dt", "B", "C")}, h0=hh))
        parts.append(p)
    # both are within their bounds of the exact scan; memories here last at most some thousand tokens
    tol = 2 ** -7 if dtype == BF else 2e-5
    scale = y.float().abs().amax()
    assert ((y.float() - torch.cat(parts).float()).abs().amax() <= tol * scale).item()
    assert ((h - hh).abs().amax() <= 2e-5 * h.abs().amax()).item()
    g = grad(d, dy.to(DEV), None, dhT.to(DEV))
    again = grad(d, dy.to(DEV), None, dhT.to(DEV))
    assert all(torch.equal(g[k], again[k]) and torch.isfinite(g[k]).all() for k in g)


def test_graph_stream_and_workspace():
    """Captured and replayed with eager work between, on another stream, with a given workspace and outputs."""
    lengths, size = [700, 5, 300], (8, 2, 64, 64)
    v, dy, dhT = make(lengths, size, BF, 17)
    d, cu, dyd, dhd = dev(v), cud(lengths), dy.to(DEV), dhT.to(DEV)
    ws = torch.empty(kda.ssm_workspace_size(d["x"], d["B"], num_seqs=3, backward=True), dtype=torch.uint8, device=DEV)
    out, hT = torch.empty_like(d["x"]), torch.empty_like(d["h0"])
    y, h = call(d, cu)
    g = grad(d, dyd, cu, dhd)

    def work():
        call(d, cu, out=out, final_state=hT, workspace=ws)
        return grad(d, dyd, cu, dhd, workspace=ws)

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = work()
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(out, y) and torch.equal(hT, h) and all(torch.equal(got[k], g[k]) for k in g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work()
    for i in range(3):
        for t in (out, hT, *got.values()):
            t.fill_(3.0)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, y) and torch.equal(hT, h) and all(torch.equal(got[k], g[k]) for k in g), i
        call(d, cu)  # eager work between replays


def test_a_short_workspace_is_refused():
    v, _, _ = make([1000], (2, 1, 16, 16), BF, 18)
    d = dev(v)
    need = kda.ssm_workspace_size(d["x"], d["B"])
    assert need > 0
    with pytest.raises(kda.KdaError):
        call(d, workspace=torch.empty(need - 1, dtype=torch.uint8, device=DEV))
