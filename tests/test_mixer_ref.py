"""The float64 definitions the GPU tests rest on, against differences and closed forms (CPU)."""
import pytest
import torch

from tests import mixer_ref as M

F8 = torch.float64


def inputs(seed=0, T=9, H=4, G=2, K=3, P=2, N=2):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, dtype=F8)
    return (r(T, H, P), r(T, H), -r(H).abs() - 0.1, r(T, G, K), r(T, G, K), r(H), r(H) * 0.3, r(N, H, K, P)), \
        [0, 4, T], r(T, H, P), r(N, H, K, P)


def test_scan_of_one_state_is_the_diagonal_recurrence():
    (x, z, A, B, C, D, bias, h0), cu, _, _ = inputs(K=1, P=1, G=4)
    d = M.softplus(z + bias)
    y, h = M.ssm(x, d, A, B, C, torch.zeros_like(D), h0, cu)
    for n in range(2):
        s = h0[n, :, 0, 0]
        for t in range(cu[n], cu[n + 1]):
            s = torch.exp(d[t] * A) * s + d[t] * B[t, :, 0] * x[t, :, 0]
            assert torch.allclose(y[t, :, 0], C[t, :, 0] * s, rtol=1e-13, atol=1e-13)
        assert torch.allclose(h[n, :, 0, 0], s, rtol=1e-13, atol=1e-13)


def test_scan_without_decay_is_linear_attention():
    (x, z, A, B, C, D, bias, h0), cu, _, _ = inputs(G=1)
    y, _ = M.ssm(x, torch.ones_like(z), torch.zeros_like(A), B, C, torch.zeros_like(D), torch.zeros_like(h0), cu)
    for a, b in zip(cu[:-1], cu[1:]):
        w = torch.tril(C[a:b, 0] @ B[a:b, 0].t())
        assert torch.allclose(y[a:b], torch.einsum("ts,shp->thp", w, x[a:b]), rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("soft", [True, False])
def test_scan_gradient_against_differences(soft):
    args, cu, dy, dhT = inputs(3)
    args = list(args)
    if not soft:
        args[1] = args[1].abs() + 1
    val = M._grads(*args, cu, dy, dhT, soft)
    names = ["dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "dh0"]
    g = torch.Generator().manual_seed(5)

    def loss(a):
        d = M.softplus(a[1] + a[6]) if soft else a[1] + a[6]
        y, h = M.ssm(a[0], d, a[2], a[3], a[4], a[5], a[7], cu)
        return (y * dy).sum() + (h * dhT).sum()

    for i, k in enumerate(names):
        v = torch.randn(args[i].shape, generator=g, dtype=F8)
        e = 1e-5
        up, dn = list(args), list(args)
        up[i], dn[i] = args[i] + e * v, args[i] - e * v
        want = ((loss(up) - loss(dn)) / (2 * e)).item()
        got = (val[k] * v).sum().item()
        assert abs(got - want) <= 1e-7 * max(1, abs(want)), (k, got, want)


def test_scan_gradient_magnitudes_are_above_the_gradient():
    args, cu, dy, dhT = inputs(4)
    val = M._grads(*args, cu, dy, dhT, True)
    mag = M.ssm_grad_mag(*args, cu, dy, dhT, True)
    for k in val:
        assert (val[k].abs() <= mag[k] * (1 + 1e-12) + 1e-12).all(), k


@pytest.mark.parametrize("name", ["silu", "sigmoid", "gelu"])
def test_gated_products_gradient_against_autograd_and_differences(name):
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, dtype=F8)
    x, wg, wu, dh = r(5, 4), r(3, 4), r(3, 4), r(5, 3)
    val, _ = M.glu(x, wg, wu, name, dh, torch.float32)
    lv = [t.clone().requires_grad_(True) for t in (x, wg, wu)]
    a = M.act(name, lv[0] @ lv[1].t())[0]
    want = torch.autograd.grad(a * (lv[0] @ lv[2].t()), lv, dh)
    for k, w in zip(("dx", "dw_gate", "dw_up"), want):
        assert torch.allclose(val[k], w, rtol=1e-12, atol=1e-12)
    z = r(50) * 4
    e = 1e-5
    slope = (M.act(name, z + e)[0] - M.act(name, z - e)[0]) / (2 * e)
    assert torch.allclose(M.act(name, z)[1], slope, rtol=1e-8, atol=1e-9)


@pytest.mark.parametrize("dtype", [torch.int8, torch.float8_e4m3fn])
def test_quantise_takes_the_nearest_value(dtype):
    g = torch.Generator().manual_seed(2)
    x = torch.randn(6, 33, generator=g)
    x[0] = 0
    x[1, 0] = 127.0 if dtype == torch.int8 else 448.0
    x[1, 1:] = torch.arange(32) + 0.5  # on borders of int8, where the scale is one
    code, scale = M.quantise(x, dtype)
    values, even = M.formats(dtype)
    for i in range(6):
        s = scale[i].double()
        if s == 0:
            assert (code[i] == 0).all()
            continue
        d = (x[i].double()[:, None] / s - values).abs()
        assert torch.equal((x[i].double() / s - code[i]).abs(), d.amin(1))
    if dtype == torch.int8:
        assert scale[1] == 1 or abs(scale[1].item() - 1) < 1e-7
        if scale[1] == 1:
            assert torch.equal(code[1, 1:] % 2, torch.zeros(32, dtype=F8))
