"""The operators around the state layer on large inputs: the kernels that read past
the last-level cache (inputs of 128 MiB and more) in every tap count, activation and
stream type, and column sums over many rows."""
import pytest
import torch

import kda_recurrent_state_amd as kda
from tests import block_ref as R
from tests.parity import log
from tests.test_gpu_block import DEV, pieces, sums_match

pytestmark = pytest.mark.gpu
F8, F4, BF = torch.float64, torch.float32, torch.bfloat16
LARGE = 128 << 20


def cuts_of(T, n):
    return [i * (T // n) for i in range(n)] + [T]


@pytest.mark.parametrize("dtype", [F4, BF])
@pytest.mark.parametrize("act", ["silu", None])
def test_gated_norm_past_the_cache(act, dtype):
    T, D = (30000, 2501) if dtype is BF else (17000, 2051)
    log(f"gated norm past the cache {act} {dtype}")
    torch.manual_seed(7)
    x, g, dy = (torch.randn(T, 1, D, device=DEV, dtype=dtype) for _ in range(3))
    w = torch.rand(D, device=DEV) + 0.5
    cuts = cuts_of(T, 4)
    inputs = 1 + (act is not None)
    assert inputs * x.nbytes >= LARGE > (inputs + 1) * x[:cuts[1]].nbytes
    kw = dict(activation=act or "sigmoid")
    gate = g if act else None
    y = kda.norm_gate_fwd(x, w, gate, **kw)
    (yh,) = pieces(lambda a, b: [kda.norm_gate_fwd(a, w, b if act else None, **kw)], cuts, x, g)
    assert torch.equal(y, yh)
    G = kda.norm_gate_bwd(x, w, dy, gate, **kw)
    parts = [kda.norm_gate_bwd(x[a:b], w, dy[a:b], g[a:b] if act else None, **kw) for a, b in zip(cuts, cuts[1:])]
    assert torch.equal(G["dx"], torch.cat([p["dx"] for p in parts]))
    if act:
        assert torch.equal(G["dgate"], torch.cat([p["dgate"] for p in parts]))
    n = x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)
    size = g.float().abs() if act else 1.0  # |g s(g)| <= |g|
    terms = (n * dy.float() * size).abs().double().sum((0, 1)) * 1.01
    sums_match(G["dweight"], [p["dweight"] for p in parts], terms)


@pytest.mark.parametrize("dtype,rdtype", [(F4, F4), (BF, BF), (BF, F4)])
def test_residual_norm_past_the_cache(dtype, rdtype):
    """With a derivative of the stream and a learned scale, which the gradient reads as well."""
    T, D = {(F4, F4): (17000, 2051), (BF, BF): (30000, 2501), (BF, F4): (20000, 2501)}[dtype, rdtype]
    log(f"residual norm past the cache {dtype} {rdtype}")
    torch.manual_seed(8)
    x, dy = (torch.randn(T, D, device=DEV, dtype=dtype) for _ in range(2))
    res, dres = (torch.randn(T, D, device=DEV, dtype=rdtype) for _ in range(2))
    w, cs = torch.rand(D, device=DEV) + 0.5, torch.rand(D, device=DEV) + 0.5
    cuts = cuts_of(T, 8)
    assert x.nbytes + res.nbytes >= LARGE > 2 * (x[:cuts[1]].nbytes + res[:cuts[1]].nbytes)
    kw = dict(scale=0.5, channel_scale=cs)
    y, h = kda.residual_norm_fwd(x, res, w, **kw)
    yh, hh = pieces(lambda a, b: kda.residual_norm_fwd(a, b, w, **kw), cuts, x, res)
    assert torch.equal(y, yh) and torch.equal(h, hh)
    inplace = res.clone()
    y, h2 = kda.residual_norm_fwd(x, inplace, w, residual_out=inplace, **kw)
    assert torch.equal(y, yh) and torch.equal(inplace, hh)
    G = kda.residual_norm_bwd(x, h, w, dy, dres, **kw)
    parts = [kda.residual_norm_bwd(x[a:b], h[a:b], w, dy[a:b], dres[a:b], **kw) for a, b in zip(cuts, cuts[1:])]
    for k in ("dx", "dresidual"):
        assert torch.equal(G[k], torch.cat([p[k] for p in parts]))
    n = h.float() * torch.rsqrt(h.float().square().mean(-1, keepdim=True) + 1e-6)
    sums_match(G["dweight"], [p["dweight"] for p in parts], (n * dy.float()).abs().double().sum(0) * 1.01)
    # dh enters the scale's sum before its rounding to the stream's type: 1.01 covers a bf16 step
    terms = (0.5 * G["dresidual"].float() * x.float()).abs().double().sum(0) * 1.01
    sums_match(G["dchannel_scale"], [p["dchannel_scale"] for p in parts], terms)


@pytest.mark.parametrize("dtype", [F4, BF])
@pytest.mark.parametrize("W,act", [(2, "silu"), (3, "silu"), (2, None), (3, None), (4, None)])
def test_conv_past_the_cache(W, act, dtype):
    C = 2504
    T = 30000 if dtype is BF else 15000
    cut = T // 2 + 1
    log(f"conv past the cache W={W} {act} {dtype}")
    torch.manual_seed(9)
    x, dy = (torch.randn(T, C, device=DEV, dtype=dtype) for _ in range(2))
    w, b = torch.randn(C, W, device=DEV) * 0.5, torch.randn(C, device=DEV)
    assert x.nbytes >= LARGE > x[:cut].nbytes
    cu = torch.tensor([0, cut, T], dtype=torch.int32, device=DEV)
    y, st = kda.conv_fwd(x, w, b, None, cu, activation=act)
    yh, sh = pieces(lambda a: kda.conv_fwd(a, w, b, activation=act), [0, cut, T], x)
    assert torch.equal(y, yh) and torch.equal(st, sh)
    G = kda.conv_bwd(x, w, dy, b, None, cu, activation=act)
    # windows at the sequences' ends and inside them, against the definition
    for beg, end in ((0, cut), (cut, T)):
        for lo in (beg, (beg + end) // 2, end - 16):
            hi = lo + 16
            first, last = max(lo - (W - 1), beg), min(hi + (W - 1), end)
            before = x[first - (W - 1):first] if first > beg else torch.zeros_like(x[:W - 1])
            f8 = [t.cpu().double() for t in (x[first:last], w, b, before[None])]
            val, bnd = R.conv(*f8, [0, last - first], act == "silu")
            sl = slice(lo - first, hi - first)
            R.check(y[lo:hi], val["y"][sl], bnd["y"][sl], "y")
            val, bnd = R.conv_grad(*f8, [0, last - first], act == "silu", dy[first:last].cpu().double(),
                                   torch.zeros(1, W - 1, C, dtype=F8))
            R.check(G["dx"][lo:hi], val["dx"][sl], bnd["dx"][sl], "dx")
    parts = [kda.conv_bwd(x[s], w, dy[s], b, activation=act) for s in (slice(0, cut), slice(cut, T))]
    # |dz| <= 1.1 |dy|, and sum |x dz| <= the product of the columns' norms
    nx, nd = x.double().square().sum(0).sqrt(), 1.1 * dy.double().square().sum(0).sqrt()
    sums_match(G["dweight"], [t["dweight"] for t in parts], (nx * nd)[:, None] * 1.01)
    sums_match(G["dbias"], [t["dbias"] for t in parts], 1.1 * dy.double().abs().sum(0) * 1.01)


# ------------------------------------------------------------------ column sums over many rows
# Whole numbers, whose sums stay below 2^24: float32 adds them exactly in any order, so a
# row that is lost or counted twice shows, and the 64-bit sum is the only right answer.
# Rows of +-1 have the norm 1 (eps 0).

def whole(g, *shape, dtype=BF, signs=False):
    t = torch.randint(0, 2, shape, generator=g, device=DEV) * 2 - 1 if signs else \
        torch.randint(-1, 2, shape, generator=g, device=DEV)
    return t.to(dtype)


@pytest.mark.parametrize("dtype", [F4, BF])
@pytest.mark.parametrize("T,H,D", [(32768, 32, 128), (65521, 3, 64), (40009, 1, 256), (5003, 1, 4096)])
def test_gated_norm_weight_gradient_over_many_rows(T, H, D, dtype):
    log(f"gated norm weight gradient {T * H} rows of {D} {dtype}")
    g = torch.Generator(device=DEV).manual_seed(10)
    x, dy = whole(g, T, H, D, dtype=dtype, signs=True), whole(g, T, H, D, dtype=dtype)
    w = whole(g, D, dtype=F4)
    got = kda.norm_gate_bwd(x, w, dy, eps=0.0)["dweight"]
    assert torch.equal(got.double(), (x.double() * dy.double()).sum((0, 1)))


@pytest.mark.parametrize("dtype,rdtype", [(F4, F4), (BF, BF), (BF, F4)])
@pytest.mark.parametrize("T,D", [(131072, 256), (30011, 1024), (9001, 8192)])
def test_residual_norm_sums_over_many_rows(T, D, dtype, rdtype):
    log(f"residual norm sums {T} rows of {D} {dtype} {rdtype}")
    g = torch.Generator(device=DEV).manual_seed(11)
    x, dy = (whole(g, T, D, dtype=dtype) for _ in range(2))
    h, dres = whole(g, T, D, dtype=rdtype, signs=True), whole(g, T, D, dtype=rdtype)
    w, cs = whole(g, D, dtype=F4), whole(g, D, dtype=F4)
    got = kda.residual_norm_bwd(x, h, w, dy, dres, scale=0.5, channel_scale=cs, eps=0.0)
    assert torch.equal(got["dweight"].double(), (h.double() * dy.double()).sum(0))
    zero = torch.zeros_like(dy)  # the sum's derivative is then the stream's
    got = kda.residual_norm_bwd(x, h, w, zero, dres, scale=0.5, channel_scale=cs, eps=0.0)
    assert torch.equal(got["dchannel_scale"].double(), 0.5 * (x.double() * dres.double()).sum(0))


@pytest.mark.parametrize("dtype", [F4, BF])
@pytest.mark.parametrize("T,C,W", [(131072, 256, 4), (65521, 1000, 3), (20011, 4096, 2), (200003, 7, 4)])
def test_conv_weight_gradient_over_many_tokens(T, C, W, dtype):
    log(f"conv weight gradient {T} x {C} W={W} {dtype}")
    g = torch.Generator(device=DEV).manual_seed(12)
    x, dy = (whole(g, T, C, dtype=dtype) for _ in range(2))
    cuts = [0, 1, T // 3, T // 3, T // 3 + 2, T]
    cu = torch.tensor(cuts, dtype=torch.int32, device=DEV)
    state = whole(g, len(cuts) - 1, W - 1, C, dtype=dtype)
    w, b = whole(g, C, W, dtype=F4), whole(g, C, dtype=F4)
    got = kda.conv_bwd(x, w, dy, b, state, cu, activation=None)
    want = torch.zeros(C, W, dtype=F8, device=DEV)
    for n, (s, e) in enumerate(zip(cuts, cuts[1:])):
        ext = torch.cat([state[n], x[s:e]]).double()
        for j in range(W):
            want[:, j] += (ext[j:j + e - s] * dy[s:e].double()).sum(0)
    assert torch.equal(got["dweight"].double(), want)
    assert torch.equal(got["dbias"].double(), dy.double().sum(0))
