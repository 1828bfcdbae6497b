"""Closer bounds for the state space scan's gradients of dt, A and dt_bias than tests/mixer_ref.py has.

The derivative of token t's log decay is the sum over pairs s < t <= r (s also the state before the first token, r also
the derivative behind the last) of the products that pass from s to r.  The kernels add products of such pairs only,
none of which another sum takes away again: a chunk's states from both sides with each other and with its tokens, pairs
of tiles, and a tile's own running sums.  So `mag` is that sum with every term's absolute value and nothing else,
a_t g_t h_{t-1} with h and g formed from absolute values, and the bound counts it as the other gradients'."""
import torch

from tests import mixer_ref as M
from tests.block_ref import F8


def log_decay_mag(x, z, A, B, C, h0, cu, dy, dhT, soft=True, scale=1.0):
    T, H, P = x.shape
    per = H // B.shape[1]
    d = M.softplus(z) if soft else z  # z with its bias
    a = torch.exp(d * A * scale)
    bh, ch = B.abs().repeat_interleave(per, 1), C.abs().repeat_interleave(per, 1)
    x, dy = x.abs(), dy.abs()
    out = torch.zeros(T, H, dtype=F8)
    for n in range(len(cu) - 1):
        h, hs = h0[n].abs(), []
        for t in range(cu[n], cu[n + 1]):
            h = a[t][:, None, None] * h
            hs.append(h)  # a_t h_{t-1}
            h = h + (d[t][:, None] * bh[t])[:, :, None] * x[t][:, None]
        g = dhT[n].abs()
        for t in reversed(range(cu[n], cu[n + 1])):
            g = g + ch[t][:, :, None] * dy[t][:, None]
            out[t] = (g * hs[t - cu[n]]).sum((1, 2))
            g = a[t][:, None, None] * g
    return out


def grad_bounds(x, z, A, B, C, D, bias, h0, cu, dy, dhT, soft=True, dtype=torch.float32):
    """mixer_ref.ssm_grad_bounds, sequence by sequence, with the closer bounds of ddt, dA and ddt_bias."""
    K, P, H = B.shape[2], x.shape[2], x.shape[1]
    R = 224 + 8 * (6 * K + 6 * P + 64 + H) + 12 * max([b - a for a, b in zip(cu[:-1], cu[1:])] + [0])
    vals, bounds = [], []
    for n in range(len(cu) - 1):
        t, T = slice(cu[n], cu[n + 1]), cu[n + 1] - cu[n]
        one = (x[t], z[t], A, B[t], C[t], D, bias, h0[n:n + 1], [0, T], dy[t], dhT[n:n + 1], soft)
        if T == 0:  # the state's derivative passes through, exactly
            zero = {"dx": x[t], "ddt": z[t], "dA": A, "dB": B[t], "dC": C[t], "dD": D, "ddt_bias": bias, "dh0": h0[n:n + 1]}
            bounds.append({k: torch.zeros_like(v) for k, v in zero.items()})
            vals.append({**bounds[-1], "dh0": dhT[n:n + 1]})
            continue
        vals.append(M._grads(*one))
        step = M.softplus(z[t] + bias) if soft else z[t] + bias
        slope = torch.sigmoid(z[t] + bias) if soft else torch.ones_like(step)
        bound = 0
        for weight, scale in ((R, 1.0), (16, 0.5)):
            m = M.ssm_grad_mag(*one, scale)
            dl = log_decay_mag(x[t], z[t] + bias, A, B[t], C[t], h0[n:n + 1], [0, T], dy[t], dhT[n:n + 1], soft, scale)
            # the derivative of a step comes through its decay and through its input
            through = m["dx"] - D.abs()[:, None] * dy[t].abs()
            dd = (through / step.clamp(min=1e-300)[..., None] * x[t].abs()).sum(-1).clamp(min=0)
            ddt = (dl * A.abs() + dd) * slope
            m.update(ddt=ddt, dA=(dl * step).sum(0), ddt_bias=ddt.sum(0))
            extra = {"dx": M.BF_OPERAND, "dB": 64, "dC": 64} if dtype != torch.float32 and scale == 1.0 else {}
            m = {k: (weight + extra.get(k, 0)) * v for k, v in m.items()}
            bound = m if bound == 0 else {k: bound[k] + m[k] for k in m}
        bounds.append(bound)
    join = lambda parts: {k: sum(p[k] for p in parts) if k in ("dA", "dD", "ddt_bias") else torch.cat([p[k] for p in parts])
                          for k in parts[0]}
    return join(vals), join(bounds)
