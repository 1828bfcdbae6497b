"""A block of a state space model run as it would be used: norm, convolution, scan, gated norm, norm, gated
feed-forward products; its gradient; its states kept in 8 bits, resumed and advanced token by token, in a
captured graph too.  Every operator's results are held to the float64 definition at the inputs that it
really had (tests/mixer_ref.py and tests/block_ref.py derive the tolerances)."""
import pytest
import torch

import kda_recurrent_state_amd as kda
from tests import block_ref as R
from tests import mixer_ref as M
from tests.parity import log

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F8, F4, BF = torch.float64, torch.float32, torch.bfloat16
LENS = [70, 0, 1, 129, 33]
H, G, K, P, W, F = 6, 2, 24, 20, 4, 152
INNER, CH = H * P, H * P + 2 * G * K
D = 72
EPS = 1e-5


def c8(t):
    return t.detach().to("cpu", F8)


class Layer:
    """Weights of one block and its parts; the projections between them are torch's."""

    def __init__(self, dtype, seed):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g)
        self.dtype = dtype
        cast = lambda t: t.to(dtype).to(DEV)
        self.norm1, self.norm2, self.norm3 = (1 + 0.1 * r(D)).to(DEV), (1 + 0.1 * r(P)).to(DEV), (1 + 0.1 * r(D)).to(DEV)
        self.w_in = cast(r(CH + H + INNER, D) / D ** 0.5)
        self.conv_w, self.conv_b = (r(CH, W) / 2).to(DEV), (0.1 * r(CH)).to(DEV)
        self.A, self.Dskip, self.bias = -(torch.rand(H, generator=g) * 8 + 1).to(DEV), r(H).to(DEV), (r(H) - 3).to(DEV)
        self.w_out = cast(r(D, INNER) / INNER ** 0.5)
        self.w_gate, self.w_up, self.w_down = cast(r(F, D) / D ** 0.5), cast(r(F, D) / D ** 0.5), cast(r(D, F) / F ** 0.5)

    def project(self, y):
        p = y @ self.w_in.t()
        return p[:, :CH], p[:, CH:CH + H].float(), p[:, CH + H:].unflatten(1, (H, P))

    def split(self, z):
        x, b, c = z.split([INNER, G * K, G * K], 1)
        return x.unflatten(1, (H, P)), b.unflatten(1, (G, K)), c.unflatten(1, (G, K))

    def mixed(self, s, dt, y, gate):
        n = kda.norm_gate_fwd(y, self.norm2, gate, activation="silu", eps=EPS)
        return n, n.flatten(1) @ self.w_out.t()

    def fed(self, o, r1):
        y2, r2 = kda.residual_norm_fwd(o, r1, self.norm3, eps=EPS)
        return y2, r2

    def ssm_args(self):
        return dict(D=self.Dskip, dt_bias=self.bias)


def held(what, pairs):
    w = [f"{k} {R.check(got, ref, bound, what + ' ' + k):.3f}" for k, got, ref, bound in pairs]
    log(f"  {what}: " + " ".join(w))


def inputs(dtype, seed):
    g = torch.Generator().manual_seed(seed)
    T, N = sum(LENS), len(LENS)
    r = lambda *s: torch.randn(*s, generator=g)
    return r(T, D).to(dtype).to(DEV), r(T, D).to(DEV), 0.3 * r(N, W - 1, CH).to(dtype).to(DEV), 0.2 * r(N, H, K, P).to(DEV)


@pytest.mark.parametrize("dtype", [F4, BF])
def test_block_forward_and_gradient(dtype):
    log(f"state space block {dtype}")
    m = Layer(dtype, 1)
    x, stream, cs0, h0 = inputs(dtype, 2)
    bounds = R.bounds_of(LENS)
    cu = torch.tensor(bounds, dtype=torch.int32, device=DEV)

    y1, r1 = kda.residual_norm_fwd(x, stream, m.norm1, eps=EPS)
    xbc, dt, gate = m.project(y1)
    z, cs = kda.conv_fwd(xbc, m.conv_w, m.conv_b, cs0, cu, activation="silu")
    xs, B, C = m.split(z)
    y, h = kda.ssm_fwd(xs, dt, m.A, B, C, h0=h0, cu_seqlens=cu, **m.ssm_args())
    n, o = m.mixed(None, dt, y, gate)
    y2, r2 = m.fed(o, r1)
    hid, saved = kda.glu_fwd_saved(y2, m.w_gate, m.w_up)
    out = hid @ m.w_down.t()
    assert torch.isfinite(out).all()

    a = [c8(t) for t in (xs, dt, m.A, B, C, m.Dskip, m.bias, h0)]
    val, bnd = M.ssm_bounds(*a, bounds, dtype=dtype)
    held("scan", [("y", y, val["y"], bnd["y"]), ("h", h, val["h"], bnd["h"])])
    val, bnd = R.conv(c8(xbc), c8(m.conv_w), c8(m.conv_b), c8(cs0), bounds, True)
    held("convolution", [("y", z, val["y"], bnd["y"])])
    val, bnd = R.norm_gate(c8(y), c8(m.norm2), c8(gate), "silu", EPS)
    held("gated norm", [("y", n, val, bnd)])
    val, bnd = R.residual_norm(c8(o), c8(r1), c8(m.norm3), 1.0, None, EPS)
    held("norm", [("y", y2, val["y"], bnd["y"]), ("residual", r2, val["residual"], bnd["residual"])])

    # backwards, from a derivative of the block's output and of the states
    g = torch.Generator().manual_seed(3)
    rand = lambda t, s=1.0: (s * torch.randn(t.shape, generator=g)).to(t.dtype).to(DEV)
    dout, dres, dh_T, dcs = rand(out), rand(r2), rand(h, 0.2), rand(cs, 0.2)
    dhid = dout @ m.w_down
    gl = kda.glu_bwd(y2, m.w_gate, m.w_up, dhid, saved=saved)
    val, bnd = M.glu(c8(y2), c8(m.w_gate), c8(m.w_up), "silu", c8(dhid), dtype)
    held("products", [("h", hid, val["h"], bnd["h"])] + [(k, gl[k], val[k], bnd[k]) for k in ("dx", "dw_gate", "dw_up")])
    n3 = kda.residual_norm_bwd(None, r2, m.norm3, gl["dx"], dres, eps=EPS)
    val, bnd = R.residual_norm_grad(c8(o), c8(r2), c8(m.norm3), 1.0, None, EPS, c8(gl["dx"]), c8(dres))
    held("norm's gradient", [(k, n3[k], val[k], bnd[k]) for k in ("dx", "dresidual", "dweight")])
    dn = (n3["dx"] @ m.w_out).unflatten(1, (H, P))
    n2 = kda.norm_gate_bwd(y, m.norm2, dn, gate, activation="silu", eps=EPS)
    val, bnd = R.norm_gate_grad(c8(y), c8(m.norm2), c8(gate), "silu", EPS, c8(dn))
    held("gated norm's gradient", [(k, n2[k], val[k], bnd[k]) for k in val])
    s = kda.ssm_bwd(xs, dt, m.A, B, C, n2["dx"], h0=h0, cu_seqlens=cu, dh_T=dh_T, **m.ssm_args())
    val, bnd = M.ssm_grad_bounds(*a, bounds, c8(n2["dx"]), c8(dh_T), dtype=dtype)
    held("scan's gradient", [(k, s[k], val[k], bnd[k]) for k in val])
    dz = torch.cat([s["dx"].flatten(1), s["dB"].flatten(1), s["dC"].flatten(1)], 1)
    cv = kda.conv_bwd(xbc, m.conv_w, dz, m.conv_b, cs0, cu, dcs, activation="silu")
    val, bnd = R.conv_grad(c8(xbc), c8(m.conv_w), c8(m.conv_b), c8(cs0), bounds, True, c8(dz), c8(dcs))
    held("convolution's gradient", [(k, cv[k], val[k], bnd[k]) for k in val])


def token(m, x, stream, codes, scales, slots, cs, ws, h):
    """One token of every sequence, the states taken from the cache and put back."""
    y1, r1 = kda.residual_norm_fwd(x, stream, m.norm1, eps=EPS)
    xbc, dt, gate = m.project(y1)
    kda.state_cache_read(codes, scales, slots, out=h)
    cs_in, h_in = cs.clone(), h.clone()
    y, cs, h = kda.ssm_conv_step(xbc, m.conv_w, cs, dt, m.A, h, m.Dskip, m.bias, m.conv_b, workspace=ws)
    kda.state_cache_write(h, codes, scales, slots)
    n, o = m.mixed(None, dt, y, gate)
    y2, r2 = m.fed(o, r1)
    hid = kda.glu_fwd(y2, m.w_gate, m.w_up)
    return dict(xbc=xbc, dt=dt, cs_in=cs_in, h_in=h_in, y=y, cs=cs, h=h, y2=y2, hid=hid, out=hid @ m.w_down.t())


@pytest.mark.parametrize("fmt", [torch.int8, torch.float8_e4m3fn])
@pytest.mark.parametrize("dtype", [F4, BF])
def test_resumed_from_a_cache(dtype, fmt):
    """A prompt's states put into the cache in 8 bits, then tokens from there: what the cache holds, and each
    token's results from what it held; a captured token replayed is the eager one, bit for bit."""
    log(f"state space block resumed {dtype} {fmt}")
    m = Layer(dtype, 4)
    x, stream, cs0, h0 = inputs(dtype, 5)
    N = len(LENS)
    cu = torch.tensor(R.bounds_of(LENS), dtype=torch.int32, device=DEV)
    y1, _ = kda.residual_norm_fwd(x, stream, m.norm1, eps=EPS)
    xbc, dt, _ = m.project(y1)
    z, cs = kda.conv_fwd(xbc, m.conv_w, m.conv_b, cs0, cu, activation="silu")
    xs, B, C = m.split(z)
    _, h = kda.ssm_fwd(xs, dt, m.A, B, C, h0=h0, cu_seqlens=cu, **m.ssm_args())
    codes, scales = kda.state_cache_empty(N + 3, (H, K, P), fmt, DEV)
    slots = torch.tensor([6, 0, 3, 1, 7], dtype=torch.int32, device=DEV)
    kda.state_cache_write(h, codes, scales, slots)
    q, sc = M.quantise(h.cpu(), fmt)
    back = kda.state_cache_read(codes, scales, slots)
    assert torch.equal(back.cpu(), (q.float() * sc[..., None]))

    g = torch.Generator().manual_seed(6)
    xt = [torch.randn(N, D, generator=g).to(dtype).to(DEV) for _ in range(5)]
    st = [torch.randn(N, D, generator=g).to(DEV) for _ in range(5)]
    ws = torch.empty(kda.ssm_conv_step_workspace_size(xbc[:N], h), dtype=torch.uint8, device=DEV)
    buf = torch.empty_like(h)
    start = [t.clone() for t in (codes.view(torch.uint8), scales, cs)]
    eager = []
    for t in range(5):
        s = token(m, xt[t], st[t], codes, scales, slots, cs, ws, buf)
        eager.append({k: v.clone() for k, v in s.items()})
        # the convolution's values enter the scan unrounded
        val, bnd = R.conv(c8(s["xbc"]), c8(m.conv_w), c8(m.conv_b), c8(s["cs_in"]), list(range(N + 1)), True)
        zx, zb, zc = m.split(val["y"])
        a = [zx, c8(s["dt"]), c8(m.A), zb, zc, c8(m.Dskip), c8(m.bias), c8(s["h_in"])]
        ref, rb = M.ssm_bounds(*a, list(range(N + 1)))
        ex, eb, ec = m.split(bnd["y"])
        d = M.softplus(c8(s["dt"]) + c8(m.bias))
        per = lambda v: v.repeat_interleave(H // G, 1)
        # a product of convolved values is off by each one's error times the other
        rest = lambda p, ep, q_, eq: p.abs() * eq + q_.abs() * ep + ep * eq * M.U
        eh = d[:, :, None, None] * rest(per(zb)[..., None], per(eb)[..., None], zx[:, :, None], ex[:, :, None])
        ey = (per(zc).abs()[..., None] * eh + per(ec)[..., None] * (ref["h"].abs() + eh * M.U)).sum(2) \
            + c8(m.Dskip).abs()[:, None] * ex
        held(f"token {t}", [("y", s["y"], ref["y"], rb["y"] + ey), ("h", s["h"], ref["h"], rb["h"] + eh)])
        val, bnd = M.glu(c8(s["y2"]), c8(m.w_gate), c8(m.w_up), "silu", torch.zeros(N, F, dtype=F8), dtype)
        held(f"token {t}", [("products", s["hid"], val["h"], bnd["h"])])

    # the same tokens from a captured graph, on a stream of its own, with eager work between the replays
    codes.view(torch.uint8).copy_(start[0]), scales.copy_(start[1]), cs.copy_(start[2])
    gx, gs = xt[0].clone(), st[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        token(m, gx, gs, codes, scales, slots, cs, ws, buf)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    codes.view(torch.uint8).copy_(start[0]), scales.copy_(start[1]), cs.copy_(start[2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = token(m, gx, gs, codes, scales, slots, cs, ws, buf)
    for t in range(5):
        gx.copy_(xt[t]), gs.copy_(st[t])
        graph.replay()
        torch.cuda.synchronize()
        for k in ("y", "cs", "h", "hid", "out"):
            assert torch.equal(got[k], eager[t][k]), (t, k)
