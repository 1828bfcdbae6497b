"""The state space scan, the gated products and the state cache where offsets pass 32 bits, with token strides far
apart, and with a workspace that captured graphs of two operators share.  Results are those of the same call on
contiguous copies, bit for bit; tests/test_gpu_ssm.py and its neighbours hold those to the definitions."""
import pytest
import torch

import kda_recurrent_state_amd as kda
from tests.parity import log

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F4, BF = torch.float32, torch.bfloat16


def rand(*s, dtype=F4, scale=1.0, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (scale * torch.randn(*s, generator=g, device=DEV)).to(dtype)


def far(t, stride):
    """t's values with tokens `stride` elements apart, behind an odd offset."""
    flat = t.flatten(1)
    store = torch.empty((t.shape[0] - 1) * stride + flat.shape[1] + 3, dtype=t.dtype, device=DEV)
    view = store[3:].as_strided((t.shape[0],) + tuple(t.shape[1:]), (stride,) + tuple(t[0].stride()), 3)
    view.copy_(t)
    return view


def ssm_inputs(T, N, H, G, K, P, dtype):
    return dict(x=rand(T, H, P, dtype=dtype, seed=1), dt=rand(T, H, seed=2), A=-rand(H, seed=3).abs() - 0.5,
                B=rand(T, G, K, dtype=dtype, seed=4), C=rand(T, G, K, dtype=dtype, seed=5), D=rand(H, seed=6),
                dt_bias=rand(H, seed=7) - 3, h0=rand(N, H, K, P, seed=8))


@pytest.mark.parametrize("stride", [(1 << 21) + 7, (1 << 22) + 1])
@pytest.mark.parametrize("dtype", [F4, BF])
def test_scan_over_far_tokens(dtype, stride):
    log(f"ssm far tokens {dtype} {stride}")
    T, N = 1100, 2
    v = ssm_inputs(T, N, 4, 2, 32, 64, dtype)
    cu = torch.tensor([0, 700, T], dtype=torch.int32, device=DEV)
    dy = rand(T, 4, 64, dtype=dtype, seed=9)
    y, h = kda.ssm_fwd(**v, cu_seqlens=cu)
    want = kda.ssm_bwd(**v, dy=dy, cu_seqlens=cu)
    for names in (("x",), ("B", "dt"), ("C",)):
        w = dict(v, **{k: far(v[k], stride) for k in names})
        y2, h2 = kda.ssm_fwd(**w, cu_seqlens=cu)
        assert torch.equal(y, y2) and torch.equal(h, h2), names
        got = kda.ssm_bwd(**w, dy=far(dy, stride) if names == ("C",) else dy, cu_seqlens=cu)
        assert all(torch.equal(got[k], want[k]) for k in want), names
        del w, got
        torch.cuda.empty_cache()


def test_scan_of_more_than_32_bits():
    """More than 2^32 bytes of x and of states kept by chunk, in many sequences of one length."""
    log("ssm 2^32 bytes")
    N, L, H, P, K = 70, 512, 64, 1024, 16
    v = ssm_inputs(N * L, N, H, 1, K, P, BF)
    assert v["x"].nbytes > 1 << 32
    v["h0"] = None
    y, h = kda.ssm_fwd(**v, num_seqs=N)
    dy = v["x"].flip(0)
    got = kda.ssm_bwd(**v, dy=dy, num_seqs=N)
    for n in (0, 33, N - 1):
        part = slice(n * L, (n + 1) * L)
        one = dict(v, **{k: v[k][part].clone() for k in ("x", "dt", "B", "C")})
        y1, h1 = kda.ssm_fwd(**one)
        # the segments a sequence is cut into depend on the whole call's size: equal but for the order of sums
        tol = lambda a, b: float((a.float() - b.float()).abs().max() / b.float().abs().max())
        assert tol(y[part], y1) < 2.0 ** -7 and tol(h[n], h1[0]) < 1e-5
        g1 = kda.ssm_bwd(**one, dy=dy[part].clone())
        assert tol(got["dx"][part], g1["dx"]) < 2.0 ** -7 and tol(got["dh0"][n], g1["dh0"][0]) < 1e-5
        assert tol(got["ddt"][part], g1["ddt"]) < 1e-5


@pytest.mark.parametrize("dtype", [F4, BF])
def test_products_over_far_tokens(dtype):
    log(f"glu far tokens {dtype}")
    T, D, F = 1100, 128, 200
    x, wg, wu = rand(T, D, dtype=dtype, seed=1), rand(F, D, dtype=dtype, seed=2), rand(F, D, dtype=dtype, seed=3)
    dh = rand(T, F, dtype=dtype, seed=4)
    for stride in ((1 << 20) + 8, (1 << 22) + 1):
        fx, fd = far(x, stride), far(dh, stride)
        assert torch.equal(kda.glu_fwd(x, wg, wu), kda.glu_fwd(fx, wg, wu))
        assert torch.equal(kda.glu_fwd(x[:40], wg, wu), kda.glu_fwd(fx[:40], wg, wu))
        a, b = kda.glu_bwd(x, wg, wu, dh), kda.glu_bwd(fx, wg, wu, fd)
        assert all(torch.equal(a[k], b[k]) for k in a)
        del fx, fd
        torch.cuda.empty_cache()


def test_products_of_more_than_32_bits():
    log("glu 2^32 bytes")
    T, D, F = 300000, 64, 8192
    x, wg, wu = rand(T, D, dtype=BF, seed=1), rand(F, D, dtype=BF, seed=2), rand(F, D, dtype=BF, seed=3)
    h, saved = kda.glu_fwd_saved(x, wg, wu)
    assert h.nbytes > 1 << 32
    at = slice(T - 500, T)
    h1, s1 = kda.glu_fwd_saved(x[at].clone(), wg, wu)
    assert torch.equal(h[at], h1) and torch.equal(saved[:, at], s1)


@pytest.mark.parametrize("fmt", [torch.int8, torch.float8_e4m3fn])
def test_cache_past_32_bits(fmt):
    log(f"state cache 2^32 bytes {fmt}")
    S, shape = 40000, (8, 128, 128)
    codes, scales = kda.state_cache_empty(S, shape, fmt, DEV)
    assert codes.nbytes > 1 << 32
    x = rand(3, *shape, seed=1)
    slots = torch.tensor([S - 1, 17, 32768], dtype=torch.int32, device=DEV)
    kda.state_cache_write(x, codes, scales, slots)
    small, sc = kda.state_cache_empty(3, shape, fmt, DEV)
    kda.state_cache_write(x, small, sc)
    at = slots.long()
    assert torch.equal(codes.view(torch.uint8)[at], small.view(torch.uint8)) and torch.equal(scales[at], sc)
    assert torch.equal(kda.state_cache_read(codes, scales, slots), kda.state_cache_read(small, sc))
    assert int((scales != 0).any(-1).any(-1).sum()) == 3


def test_graphs_that_share_a_workspace():
    log("graphs that share a workspace")
    v = ssm_inputs(900, 3, 4, 2, 32, 40, BF)
    cu = torch.tensor([0, 1, 600, 900], dtype=torch.int32, device=DEV)
    dy = rand(900, 4, 40, dtype=BF, seed=9)
    x, wg, wu, dh = rand(130, 100, seed=1), rand(70, 100, seed=2), rand(70, 100, seed=3), rand(130, 70, seed=4)
    need = max(kda.ssm_workspace_size(v["x"], v["B"], num_seqs=3, backward=True),
               kda.glu_workspace_size(x, wg, wu, backward=True))
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device=DEV)
    scan = lambda: kda.ssm_bwd(**v, dy=dy, cu_seqlens=cu, workspace=ws)
    products = lambda: kda.glu_bwd(x, wg, wu, dh, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        scan(), products()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(ga):
        a = scan()
    with torch.cuda.graph(gb):
        b = products()
    for i in range(4):
        dy.copy_(rand(900, 4, 40, dtype=BF, seed=20 + i))
        dh.copy_(rand(130, 70, seed=30 + i))
        for g in ((ga, gb), (gb, ga))[i % 2]:
            g.replay()
        torch.cuda.synchronize()
        ea, eb = kda.ssm_bwd(**v, dy=dy, cu_seqlens=cu), kda.glu_bwd(x, wg, wu, dh)
        assert all(torch.equal(a[k], ea[k]) for k in ea) and all(torch.equal(b[k], eb[k]) for k in eb)
