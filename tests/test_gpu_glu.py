"""The gated feed-forward products on the GPU against their float64 definition (tests/mixer_ref.py, which
also derives the tolerances)."""
import pytest
import torch

import kda_recurrent_state_amd as kda
from tests import mixer_ref as M
from tests.parity import log

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F4, BF = torch.float32, torch.bfloat16
# tokens, width, hidden: one token and few, across the few/tiled rule, whole tiles, odd everything
SIZES = [(1, 64, 64), (3, 17, 5), (16, 256, 48), (33, 100, 70), (64, 64, 130), (65, 64, 64), (130, 192, 200), (77, 1, 1),
         (300, 100, 270), (257, 64, 129), (1, 1000, 333), (512, 128, 384)]


def make(size, dtype, seed=1):
    T, D, F = size
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    return r(T, D).to(dtype), (r(F, D) * D ** -0.5).to(dtype), (r(F, D) * D ** -0.5).to(dtype), r(T, F).to(dtype)


def slice_of(t):
    wide = torch.full((t.shape[0], 3, t.shape[1]), 7.0, dtype=t.dtype, device=t.device)
    wide[:, 1] = t
    return wide[:, 1]


@pytest.mark.parametrize("dtype", [F4, BF])
@pytest.mark.parametrize("act", ["silu", "sigmoid", "gelu"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_against_definition(size, act, dtype):
    log(f"glu {size} {act} {dtype}")
    x, wg, wu, dh = make(size, dtype)
    val, bnd = M.glu(x.double(), wg.double(), wu.double(), act, dh.double(), dtype)
    x, wg, wu, dh = (t.to(DEV) for t in (x, wg, wu, dh))
    h = kda.glu_fwd(x, wg, wu, activation=act)
    w = [M.check(h, val["h"], bnd["h"], "h")]
    h2, saved = kda.glu_fwd_saved(x, wg, wu, activation=act)
    assert torch.equal(h, h2)
    a, b = kda.glu_bwd(x, wg, wu, dh, activation=act), kda.glu_bwd(x, wg, wu, dh, activation=act, saved=saved)
    for k in ("dx", "dw_gate", "dw_up"):
        w += [M.check(a[k], val[k], bnd[k], k), M.check(b[k], val[k], bnd[k], k + " from saved")]
    # slices of wider rows, halves of one weight, which lie elsewhere in memory
    both = torch.cat([wg, wu])
    s = (slice_of(x), both[:size[2]], both[size[2]:])
    assert torch.equal(kda.glu_fwd(*s, activation=act), h)
    c = kda.glu_bwd(*s, slice_of(dh), activation=act)
    assert all(torch.equal(c[k], a[k]) for k in a)
    d = kda.glu_bwd(x, wg, wu, dh, activation=act, saved=saved, input_grad=False)
    assert d["dx"] is None and torch.equal(d["dw_gate"], b["dw_gate"]) and torch.equal(d["dw_up"], b["dw_up"])
    log("  share of the allowed error: " + " ".join(f"{v:.3f}" for v in w))


@pytest.mark.parametrize("size", [(2000, 256, 4096), (5000, 1088, 1000), (4096, 512, 8192), (4090, 4096, 72), (4090, 4000, 40),
                                  (100, 4096, 2040), (65, 4000, 2040), (50, 192, 6144)], ids=str)
def test_large_tiles(size):
    """The large tiles' shapes, in whole numbers: sums below 2^24 are exact in any order, so the weights' gradients and
    the products are too."""
    T, D, F = size
    g = torch.Generator().manual_seed(3)
    i = lambda lo, hi, *s: torch.randint(lo, hi + 1, s, generator=g).float()
    x, wg, wu = i(-2, 2, T, D).to(BF).to(DEV), i(-1, 1, F, D).to(BF).to(DEV), i(-1, 1, F, D).to(BF).to(DEV)
    h, saved = kda.glu_fwd_saved(x, wg, wu, activation="sigmoid")
    assert torch.equal(saved[0], x.float() @ wg.float().t()) and torch.equal(saved[1], x.float() @ wu.float().t())
    want = torch.sigmoid(saved[0].double()) * saved[1].double()
    assert ((h.double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-5 * saved[1].abs()).all()
    # with u = 0 and a gate of 0 the derivatives are dh / 4 * u and dh / 2: whole numbers again
    zero = torch.zeros_like(saved)
    zero[1] = i(-3, 3, T, F).to(DEV)
    dh = (4 * i(-1, 1, T, F)).to(BF).to(DEV)
    got = kda.glu_bwd(x, wg, wu, dh, activation="sigmoid", saved=zero)
    dg, du = dh.double() * zero[1].double() / 4, dh.double() / 2
    for k, want in (("dx", dg @ wg.double() + du @ wu.double()), ("dw_gate", dg.t() @ x.double()),
                    ("dw_up", du.t() @ x.double())):
        assert torch.equal(got[k], want.to(BF)), k


@pytest.mark.parametrize("dtype", [F4, BF])
def test_large_gates(dtype):
    """Gates far out on both sides: values and slopes neither overflow nor lose their sign's side."""
    x = torch.tensor([[1.0]], dtype=dtype).repeat(70, 1)
    gates = torch.tensor([-100.0, -88.5, -60.0, -17.0, -4.0, 0.0, 4.0, 17.0, 60.0, 100.0])
    wg, wu = gates[:, None].to(dtype), torch.full((10, 1), 2.0, dtype=dtype)
    dh = torch.ones(70, 10, dtype=dtype)
    for act in ("silu", "sigmoid", "gelu"):
        val, bnd = M.glu(x.double(), wg.double(), wu.double(), act, dh.double(), dtype)
        t = [v.to(DEV) for v in (x, wg, wu)]
        M.check(kda.glu_fwd(*t, activation=act), val["h"], bnd["h"], act)
        got = kda.glu_bwd(*t, dh.to(DEV), activation=act)
        for k in got:
            M.check(got[k], val[k], bnd[k], f"{act} {k}")


def test_no_tokens():
    x, wg, wu, dh = (t.to(DEV) for t in make((4, 64, 32), BF))
    assert kda.glu_fwd(x[:0], wg, wu).shape == (0, 32)
    got = kda.glu_bwd(x[:0], wg, wu, dh[:0])
    assert got["dx"].shape == (0, 64) and not got["dw_gate"].any() and not got["dw_up"].any()


@pytest.mark.parametrize("dtype", [F4, BF])
def test_a_row_with_nan_stays_a_row(dtype):
    x, wg, wu, _ = (t.to(DEV) for t in make((100, 64, 70), dtype))
    h = kda.glu_fwd(x, wg, wu)
    x[7, 3] = float("nan")
    h2 = kda.glu_fwd(x, wg, wu)
    keep = torch.arange(100, device=DEV) != 7
    assert torch.equal(h[keep], h2[keep]) and torch.isnan(h2[7]).all()


@pytest.mark.parametrize("dtype,size", [(BF, (300, 128, 192)), (F4, (100, 100, 70)), (BF, (8, 128, 64))], ids=str)
def test_graph_stream_and_workspace(dtype, size):
    x, wg, wu, dh = (t.to(DEV) for t in make(size, dtype))
    h, saved = kda.glu_fwd_saved(x, wg, wu)
    g = kda.glu_bwd(x, wg, wu, dh, saved=saved)
    need = max(kda.glu_workspace_size(x, wg, wu), kda.glu_workspace_size(x, wg, wu, backward=True))
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    out, keep = torch.empty_like(h), torch.empty_like(saved)

    def work():
        kda.glu_fwd_saved(x, wg, wu, out=out, saved=keep, workspace=ws)
        return kda.glu_bwd(x, wg, wu, dh, saved=keep, workspace=ws)

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = work()
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(out, h) and all(torch.equal(got[k], g[k]) for k in g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work()
    for i in range(3):
        for t in (out, keep, *got.values()):
            t.fill_(3.0)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, h) and torch.equal(keep, saved) and all(torch.equal(got[k], g[k]) for k in g), i
        kda.glu_fwd(x, wg, wu)


def test_a_short_workspace_is_refused():
    x, wg, wu, dh = (t.to(DEV) for t in make((100, 64, 64), BF))
    need = kda.glu_workspace_size(x, wg, wu, backward=True)
    with pytest.raises(kda.KdaError):
        kda.glu_bwd(x, wg, wu, dh, workspace=torch.empty(need - 1, dtype=torch.uint8, device=DEV))
