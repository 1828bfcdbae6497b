"""Plain float64 definitions of the state space scan, the gated feed-forward products and the 8-bit state
cache, with the error bounds the GPU tests hold the kernels to (in units of u = 2^-24; a result stored in a
type with half step e adds e |value|, as in block_ref).

Scan.  A result is a sum of products, each of inputs, steps d and decays; `mag` is the same sum with every
term's absolute value.  What may be off, relative to a term:
  d              softplus by a library exponential and logarithm: 8 u
  decays         of total log |L|: d's error and the rounding of the exponent, 10 |L| u, and 4 u an
                 exponential, of which a term meets 4 (into its chunk's end, chunks and segments between,
                 into its own): (10 |L| + 16) u.  As L e^-L <= 0.74 e^-(L / 2), the part with L is at most
                 7.4 u times the same sum with half the decay.
  parts          a value in three bf16 parts is held to 2^-26; products of parts below 2^-24 left out: 4 u.
  bf16 results   y and dx are sums of products with the masked weights (C . B) decay d, and with the state; both
                 are held in fp32 and rounded once to bf16 as operands.
                 Each term of the sum has one of them as a factor, so it is off by at most half a
                 step of bf16, 2^-8 = 2^16 u, relative: 2^16 mag in all, whatever the number of terms.  dB's and dC's
                 masked weights go in as two parts, which hold them to 2^-18 = 64 u.  States, dt, A, D and
                 h0's gradients do not pass such a rounding.
  sums           one rounding an addition.  A chunk adds 32 products in each of 6 instructions to a state
                 tile: 192 roundings in a chunk of 32 tokens (fp32), the same in 64 (bf16): at most 6 u a
                 token.  A result adds K state rows (6 products each in fp32) and a chunk's 64 tokens;
                 sums over columns (P) and heads come on top in the gradient.
So bound = (R + 6 T) mag + 8 mag(half the decay), R = 128 + 64 + 32 + 8 (sums of what the result adds).
"""
import math

import torch

from tests.block_ref import F8, HALF, U, check  # noqa: F401


def softplus(z):
    return torch.clamp(z, min=0) + torch.log1p(torch.exp(-z.abs()))


def ssm(x, dt, A, B, C, D, h0, cu):
    """y and final states, token by token; dt after its softplus, all float64, differentiable."""
    T, H, P = x.shape
    per = H // B.shape[1]
    ys, hs = [], []
    for n in range(len(cu) - 1):
        h = h0[n]
        for t in range(cu[n], cu[n + 1]):
            b, c = B[t].repeat_interleave(per, 0), C[t].repeat_interleave(per, 0)
            h = torch.exp(dt[t] * A)[:, None, None] * h + (dt[t][:, None] * b)[:, :, None] * x[t][:, None]
            ys.append((c[:, :, None] * h).sum(1) + D[:, None] * x[t])
        hs.append(h)
    return (torch.stack(ys) if ys else torch.zeros(0, H, P, dtype=F8)), torch.stack(hs)


BF_OPERAND = 2.0 ** 16  # half a step of bf16 in units of u


def ssm_bounds(x, z, A, B, C, D, bias, h0, cu, soft=True, dtype=torch.float32):
    """Values and bounds of y and h_T; dtype is that of x."""
    d = softplus(z + bias) if soft else z + bias
    y, h = ssm(x, d, A, B, C, D, h0, cu)
    K, T = B.shape[2], max([b - a for a, b in zip(cu[:-1], cu[1:])] + [0])
    m = [v.abs() for v in (x, B, C, D, h0)]
    full = ssm(m[0], d, A, m[1], m[2], m[3], m[4], cu)
    half = ssm(m[0], d, A / 2, m[1], m[2], m[3], m[4], cu)
    R = 224 + 8 * (6 * K + 64) + 6 * T
    return {"y": y, "h": h}, {"y": R * full[0] + 8 * half[0], "h": R * full[1] + 8 * half[1]} \
        if dtype == torch.float32 else \
        {"y": (R + BF_OPERAND) * full[0] + 8 * half[0], "h": R * full[1] + 8 * half[1]}


def _grads(x, z, A, B, C, D, bias, h0, cu, dy, dhT, soft, scale=1.0):
    leaves = [t.clone().requires_grad_(True) for t in (x, z, A, B, C, D, bias, h0)]
    x, z, A, B, C, D, bias, h0 = leaves
    d = softplus(z + bias) if soft else z + bias
    y, h = ssm(x, d, A * scale, B, C, D, h0, cu)
    got = torch.autograd.grad([y, h], leaves, [dy, dhT], allow_unused=True)
    return dict(zip(("dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "dh0"),
                    (torch.zeros_like(l) if g is None else g for l, g in zip(leaves, got))))


def ssm_grad_mag(x, z, A, B, C, D, bias, h0, cu, dy, dhT, soft, scale=1.0):
    """The gradient's sums with every term's absolute value, by the recurrence run backwards: the parts of the derivative
    of a step that come through its decay and through its input have opposite signs and are added here."""
    T, H, P = x.shape
    G, K = B.shape[1:]
    per = H // G
    d = softplus(z + bias) if soft else z + bias
    a = torch.exp(d * A * scale)
    bh, ch = B.abs().repeat_interleave(per, 1), C.abs().repeat_interleave(per, 1)
    x, dy = x.abs(), dy.abs()
    out = {"dx": torch.zeros(T, H, P, dtype=F8), "dl": torch.zeros(T, H, dtype=F8), "dd": torch.zeros(T, H, dtype=F8),
           "dB": torch.zeros(T, H, K, dtype=F8), "dC": torch.zeros(T, H, K, dtype=F8), "dh0": torch.zeros_like(h0)}
    for n in range(len(cu) - 1):
        h, hs = h0[n].abs(), []
        for t in range(cu[n], cu[n + 1]):
            hs.append(h)
            h = a[t][:, None, None] * h + (d[t][:, None] * bh[t])[:, :, None] * x[t][:, None]
        hs.append(h)
        g = dhT[n].abs()
        for t in reversed(range(cu[n], cu[n + 1])):
            i = t - cu[n]
            g = g + ch[t][:, :, None] * dy[t][:, None]
            out["dC"][t] = (hs[i + 1] * dy[t][:, None]).sum(-1)
            out["dB"][t] = (g * (d[t][:, None] * x[t])[:, None]).sum(-1)
            dxd = (g * bh[t][:, :, None]).sum(1)
            out["dx"][t] = d[t][:, None] * dxd + D.abs()[:, None] * dy[t]
            out["dd"][t] = (dxd * x[t]).sum(-1)
            # the kernel forms this as sums of row and column sums of the chunk: both are inside these magnitudes
            out["dl"][t] = (g * hs[i + 1]).sum((1, 2)) + (g * hs[i]).sum((1, 2))
            g = a[t][:, None, None] * g
        out["dh0"][n] = g
    s = torch.sigmoid(z + bias) if soft else torch.ones_like(z)
    ddt = (out["dl"] * A.abs() + out["dd"]) * s
    return {"dx": out["dx"], "ddt": ddt, "dA": (out["dl"] * d).sum(0),
            "dB": out["dB"].view(T, G, per, K).sum(2), "dC": out["dC"].view(T, G, per, K).sum(2),
            "dD": (x * dy).sum((0, 2)), "ddt_bias": ddt.sum(0), "dh0": out["dh0"]}


def ssm_grad_bounds(x, z, A, B, C, D, bias, h0, cu, dy, dhT, soft=True, dtype=torch.float32):
    val = _grads(x, z, A, B, C, D, bias, h0, cu, dy, dhT, soft)
    full = ssm_grad_mag(x, z, A, B, C, D, bias, h0, cu, dy, dhT, soft)
    half = ssm_grad_mag(x, z, A, B, C, D, bias, h0, cu, dy, dhT, soft, 0.5)
    K, P, H = B.shape[2], x.shape[2], x.shape[1]
    T = max([b - a for a, b in zip(cu[:-1], cu[1:])] + [0])
    # both states of a chunk meet (12 T); sums over K, P, a chunk and the group's heads; a chunk's sums of rows and
    # columns are added over up to 64 tokens, each of at most the magnitude of a neighbour's in the chunk
    R = 224 + 8 * (6 * K + 6 * P + 64 + H) + 12 * T
    bound = {}
    for k in val:
        bound[k] = R * full[k] + 16 * half[k]
        if dtype != torch.float32 and k in ("dx", "dB", "dC"):
            bound[k] = bound[k] + (BF_OPERAND if k == "dx" else 64) * full[k]
    # The derivative of a log decay is a sum over pairs of tokens around it, formed as running sums of the chunk's
    # row and column sums, in which every other pair cancels: the same products are in both, but the additions
    # and factors behind them (64 + 16 roundings of a row's, of a column's sum) are not.
    bound["ddt"] = bound["ddt"] + 160 * near(full["ddt"], cu)
    for k in ("dA", "ddt_bias"):
        bound[k] = bound[k] + 160 * (near(full["ddt"], cu) * (1 if k == "ddt_bias" else
                                     (softplus(z + bias) if soft else z + bias) / A.abs().clamp(min=1e-30))).sum(0)
    return val, bound


def near(v, cu, reach=64):
    """The sum of v over the tokens of the same sequence within `reach`."""
    out = torch.zeros_like(v)
    for n in range(len(cu) - 1):
        for t in range(cu[n], cu[n + 1]):
            out[t] = v[max(cu[n], t - reach):min(cu[n + 1], t + reach + 1)].sum(0)
    return out


# ------------------------------------------------------------------ gated products

def act(name, z):
    if name == "gelu":
        cdf = 0.5 * torch.special.erfc(-z * math.sqrt(0.5))
        return z * cdf, cdf + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    s, sn = torch.sigmoid(z), torch.sigmoid(-z)
    return (z * s, s * (1 + z * sn)) if name == "silu" else (s, s * sn)


def glu(x, wg, wu, name, dh, dtype):
    """Values and bounds of h and its gradient.  A product over D adds D terms (6 D from fp32, whose terms are
    within 4 u): e = (D + 8) u mag, (6 D + 16) u mag.  The activations' slopes are at most 1.13 and their
    curvatures at most 1; they are computed within (|g| + 12) u, relative for the logistic function and
    absolute for the slopes, whose terms are at most 1 + |g|.  dg and du are rounded to bf16 where
    the inputs are."""
    T, D = x.shape
    F = wg.shape[0]
    bf = dtype == torch.bfloat16
    n = (lambda k: (k + 8) if bf else (6 * k + 16))
    g, u = x @ wg.t(), x @ wu.t()
    eg, eu = n(D) * (x.abs() @ wg.abs().t()), n(D) * (x.abs() @ wu.abs().t())
    a, s = act(name, g)
    ea, es = 1.13 * eg + (g.abs() + 12) * a.abs() + 12 * U, eg + (g.abs() + 12) * (1 + g.abs())
    val = {"h": a * u}
    bnd = {"h": a.abs() * eu + u.abs() * ea + 4 * val["h"].abs() + ea * eu * U}
    dg, du = dh * u * s, dh * a
    edg = dh.abs() * (u.abs() * es + s.abs() * eu + es * eu * U) + 4 * dg.abs()
    edu = dh.abs() * ea + 4 * du.abs()
    if bf:
        half = HALF[torch.bfloat16] / U
        edg, edu = edg + half * (dg.abs() + edg * U), edu + half * (du.abs() + edu * U)
    # a share of the sum more or less: its partial results are added too
    val["dx"] = dg @ wg + du @ wu
    bnd["dx"] = edg @ wg.abs() + edu @ wu.abs() + (n(2 * F) + 64) * (dg.abs() @ wg.abs() + du.abs() @ wu.abs())
    for k, v, e in (("dw_gate", dg, edg), ("dw_up", du, edu)):
        val[k] = v.t() @ x
        bnd[k] = e.t() @ x.abs() + (n(T) + 64) * (v.abs().t() @ x.abs())
    return val, bnd


# ------------------------------------------------------------------ state cache

def formats(dtype):
    """The format's finite values in order, and whether each one's code is even."""
    if dtype == torch.int8:
        v = torch.arange(-127, 128, dtype=F8)
        return v, v % 2 == 0
    codes = torch.arange(256, dtype=torch.uint8)
    v = codes.view(torch.float8_e4m3fn).double()
    keep = torch.isfinite(v) & ~((v == 0) & (codes == 128))
    order = torch.argsort(v[keep])
    return v[keep][order], (codes[keep][order] % 2 == 0)


def quantise(x, dtype):
    """(codes as the values they stand for, scales float32) of finite float32 rows, in exact arithmetic but for the
    scale's own definition."""
    unit = torch.tensor(1.0 / 127 if dtype == torch.int8 else 1.0 / 448, dtype=torch.float32)
    scale = x.abs().amax(-1) * unit
    values, even = formats(dtype)
    mid = (values[1:] + values[:-1]) / 2
    q = x.double() / torch.where(scale > 0, scale, torch.ones_like(scale)).double()[..., None]
    i = torch.bucketize(q, mid)
    up = (i < len(mid)) & (q == mid[i.clamp(max=len(mid) - 1)]) & ~even[i]
    return torch.where(scale[..., None] > 0, values[i + up], torch.zeros_like(q)), scale
