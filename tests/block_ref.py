"""Plain float64 definitions of the operators around the state layer, token by
token, with the error bounds the GPU tests hold the kernels to.

Every function takes CPU float64 tensors and returns values together with a
bound on what fp32 arithmetic may be off by, in units of u = 2^-24 (half a step
of fp32, relative).  The bounds are derived as follows; a result stored in a
type with half step e adds e |value|.

  exponentials   e^x is computed as 2^(x log2 e): the product's rounding is an
                 absolute error |x| u / ln 2 * ln 2 = |x| u in the result's
                 exponent, the instruction adds one unit in the last place
                 (2 u): relative error (|x| + 3) u.  The logistic function adds
                 a sum (u) and a reciprocal (2 u): (|x| + 6) u relative, and no
                 more in absolute terms for 1 - s.
  sums           n terms added in any order: (n - 1) u sum|terms| at most; the
                 kernels add in chains of at most CHAIN terms (lanes, strips,
                 workgroups and partial rows each in turn).
"""
import torch

U = 2.0 ** -24
CHAIN = 256  # longest chain of additions behind a column sum at the tests' sizes
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
F8 = torch.float64


def check(got, ref, bound_u, what):
    """|got - ref| <= half a step of got's type + bound_u * u, everywhere."""
    g = got.detach().to("cpu", F8)
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    assert torch.isfinite(g).all(), f"{what}: non-finite values"
    allowed = HALF[got.dtype] * (ref.abs() + bound_u * U) + bound_u * U + 1e-40
    over = ((g - ref).abs() / allowed)
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} times what rounding allows"
    return worst


def bounds_of(lengths):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    return cu


# ------------------------------------------------------------------ diagonal recurrence
# With mag_t = a mag_{t-1} + |x_t|, each step multiplies by an a whose relative
# error is (|log a| + 3) u, rounds a product and a sum, and the joins between
# runs of tokens round up to three times more per token: the error follows
# err_t = a (err_{t-1} + (|log a| + 3) u mag_{t-1}) + 4 u mag_t.

def scan(x, la, h0, cu):
    T, C = x.shape
    a = torch.exp(la)
    y, e = torch.zeros(T, C, dtype=F8), torch.zeros(T, C, dtype=F8)
    hT, eT = h0.clone(), torch.zeros_like(h0)
    before, ebefore = torch.zeros(T, C, dtype=F8), torch.zeros(T, C, dtype=F8)
    mbefore = torch.zeros(T, C, dtype=F8)
    for n in range(len(cu) - 1):
        h, m, er = h0[n], h0[n].abs(), torch.zeros(C, dtype=F8)
        for t in range(cu[n], cu[n + 1]):
            before[t], ebefore[t], mbefore[t] = h, er, m
            da = torch.where(a[t] > 0, la[t].abs() + 3, torch.zeros_like(a[t]))
            da = torch.nan_to_num(da, posinf=0.0)
            er = a[t] * (er + da * m)
            h, m = a[t] * h + x[t], a[t] * m + x[t].abs()
            er = er + 4 * m
            y[t], e[t] = h, er
        hT[n], eT[n] = h, er
    return dict(y=y, h=hT, before=before), dict(y=e, h=eT, before=ebefore, mag=mbefore)


def scan_grad(x, la, h0, cu, dy, dhT):
    """dx, dlog_a, dh0 and their bounds."""
    fwd, fe = scan(x, la, h0, cu)
    T, C = x.shape
    a = torch.exp(la)
    dx, ex = torch.zeros(T, C, dtype=F8), torch.zeros(T, C, dtype=F8)
    dl, el = torch.zeros(T, C, dtype=F8), torch.zeros(T, C, dtype=F8)
    dh0, e0 = dhT.clone(), torch.zeros_like(dhT)
    for n in range(len(cu) - 1):
        c, m, er = dhT[n], dhT[n].abs(), torch.zeros(C, dtype=F8)
        for t in reversed(range(cu[n], cu[n + 1])):
            g, m = dy[t] + c, dy[t].abs() + m
            er = er + 2 * m
            dx[t], ex[t] = g, er
            da = torch.nan_to_num(torch.where(a[t] > 0, la[t].abs() + 3, torch.zeros_like(a[t])), posinf=0.0)
            c, er, m = a[t] * g, a[t] * (er + (da + 2) * m), a[t] * m
            dl[t] = c * fwd["before"][t]
            el[t] = er * fe["mag"][t] + m * fe["before"][t] + 2 * m * fe["mag"][t]
        dh0[n], e0[n] = c, er
    return dict(dx=dx, dlog_a=dl, dh0=dh0), dict(dx=ex, dlog_a=el, dh0=e0)


# ------------------------------------------------------------------ short convolution
# z sums W + 1 terms: (W + 1) u M, M = |b| + sum |w x|.  SiLU's slope is at most
# 1.1 and its logistic factor is (|z| + 6) u off: y is within
# (1.1 (W + 1) + |z| + 8) M u, so (M + 14) M u.

def _act(z, silu):
    return z / (1 + torch.exp(-z)) if silu else z


def _slope(z, silu):
    s = 1 / (1 + torch.exp(-z))
    return s * (1 + z * (1 - s)) if silu else torch.ones_like(z)


def conv(x, w, b, state, cu, silu):
    T, C = x.shape
    W = w.shape[1]
    z, M = torch.zeros(T, C, dtype=F8), torch.zeros(T, C, dtype=F8)
    sT = torch.zeros_like(state)
    for n in range(len(cu) - 1):
        ext = torch.cat([state[n], x[cu[n]:cu[n + 1]]])
        for t in range(cu[n], cu[n + 1]):
            p = t - cu[n]
            z[t], M[t] = b, b.abs()
            for j in range(W):
                z[t] += w[:, j] * ext[p + j]
                M[t] += (w[:, j] * ext[p + j]).abs()
        sT[n] = ext[cu[n + 1] - cu[n]:]
    return dict(y=_act(z, silu), state=sT), dict(y=(M + 14) * M, z=z, M=M)


# dz = dy act'(z): the slope changes by at most 0.5 err_z and is computed within
# (2 |z| + 16) u: (3 M + 20) u |dy|.  dx sums W such terms times w and one of
# dstate_T; dw and db are column sums.

def conv_grad(x, w, b, state, cu, silu, dy, dsT):
    f, fe = conv(x, w, b, state, cu, silu)
    W = w.shape[1]
    dz, k = dy * _slope(fe["z"], silu), (3 * fe["M"] + 20) * dy.abs()
    dx, ex = torch.zeros_like(x), torch.zeros_like(x)
    ds, es = torch.zeros_like(state), torch.zeros_like(state)
    dw, ew = torch.zeros_like(w), torch.zeros_like(w)
    for n in range(len(cu) - 1):
        s, e = cu[n], cu[n + 1]
        L = e - s
        ext = torch.cat([state[n], x[s:e]])
        dext, eext = torch.zeros_like(ext), torch.zeros_like(ext)
        for j in range(W):
            dext[j:j + L] += w[:, j] * dz[s:e]
            eext[j:j + L] += w[:, j].abs() * (k[s:e] + (W + 2) * 1.1 * dy[s:e].abs())
            dw[:, j] += (ext[j:j + L] * dz[s:e]).sum(0)
            ew[:, j] += (ext[j:j + L].abs() * (k[s:e] + CHAIN * 1.1 * dy[s:e].abs())).sum(0)
        dext[L:] += dsT[n]
        eext[L:] += (W + 2) * dsT[n].abs()
        ds[n], es[n] = dext[:W - 1], eext[:W - 1]
        dx[s:e], ex[s:e] = dext[W - 1:], eext[W - 1:]
    T = cu[-1]
    return (dict(dx=dx, dweight=dw, dbias=dz[:T].sum(0), dstate=ds),
            dict(dx=ex, dweight=ew, dbias=(k + CHAIN * 1.1 * dy.abs())[:T].sum(0), dstate=es))


# ------------------------------------------------------------------ norms
# The mean of squares is a sum of positive terms in chains of at most 32 plus
# the lanes' tree and the wavefronts' chain (< 48 terms in all): r is within
# 24 u + 4 u, the products with w and the gate's factor add (|g| + 10) u:
# (|g| + 40) u |y|.

def _gate(g, act):
    s = 1 / (1 + torch.exp(-g))
    return (g * s, s * (1 + g * (1 - s))) if act == "silu" else (s, s * (1 - s))


def norm_gate(x, w, g, act, eps):
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    y = x * r * w
    k = 40.0
    if g is not None:
        y = y * _gate(g, act)[0]
        k = g.abs() + 40
    return y, k * y.abs()


# dx = r (d - x k), k = r^2 mean(d x): the terms' factors are within
# (|g| + 48) u each and the mean's chain adds 48 u of its absolute terms, so
# 2 (|g|max + 64) u of |r d| + |r x| r^2 mean|d x|.  dg: factors within
# (|g| + 64) u of |dy n w| (1 + |g| / 4), the slope's absolute size.  dw: a
# column sum of terms within (|g| + 64) u.

def norm_gate_grad(x, w, g, act, eps, dy):
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    n = x * r
    a, slope = _gate(g, act) if g is not None else (torch.ones_like(x), None)
    ga = g.abs() if g is not None else torch.zeros_like(x)
    d = dy * a * w
    dx = r * (d - n * (d * n).mean(-1, keepdim=True))
    gm = ga.amax(-1, keepdim=True)
    ex = 2 * (gm + 64) * ((r * d).abs() + (n * r).abs() * (d * n).abs().mean(-1, keepdim=True))
    val, bnd = dict(dx=dx), dict(dx=ex)
    if g is not None:
        val["dgate"] = dy * n * w * slope
        bnd["dgate"] = (ga + 64) * (dy * n * w).abs() * (1 + ga / 4)
    term = dy * a * n
    val["dweight"] = term.flatten(0, -2).sum(0)
    bnd["dweight"] = ((ga + 64 + CHAIN) * term.abs()).flatten(0, -2).sum(0)
    return val, bnd


# h rounds a product and a sum: 3 u (|res| + |s x|) =: 3 u M, and enters y times
# r w once directly and once through the mean: 3 u M |r w| + 3 u |y| M/|h| taken
# over the row, bounded by the row's largest; on top the norm's own 40 u |y|.

def residual_norm(x, res, w, scale, cs, eps):
    s = scale * (cs if cs is not None else torch.ones_like(w))
    h, M = res + s * x, res.abs() + (s * x).abs()
    r = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    y = h * r * w
    through = (h.abs() * M).mean(-1, keepdim=True) * r * r  # relative change of r per unit of M's error
    return dict(y=y, residual=h), dict(y=(40 + 4 * through) * y.abs() + 4 * M * (r * w).abs(), residual=4 * M)


def residual_norm_grad(x, h, w, scale, cs, eps, dy, dres):
    s = scale * (cs if cs is not None else torch.ones_like(w))
    r = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    n, d = h * r, dy * w
    dh = r * (d - n * (d * n).mean(-1, keepdim=True)) + dres
    e = 128 * ((r * d).abs() + (n * r).abs() * (d * n).abs().mean(-1, keepdim=True)) + 2 * dres.abs()
    val = dict(dx=s * dh, dresidual=dh, dweight=(dy * n).sum(0))
    bnd = dict(dx=s.abs() * (e + 3 * dh.abs()), dresidual=e, dweight=((64 + CHAIN) * (dy * n).abs()).sum(0))
    if cs is not None:
        val["dchannel_scale"] = (scale * dh * x).sum(0)
        bnd["dchannel_scale"] = (abs(scale) * x.abs() * (e + (CHAIN + 4) * dh.abs())).sum(0)
    return val, bnd
