"""The operators around the gated delta-rule state layer, as measured cases.

Four operators of a recurrent token-mixing block, each in the directions a user runs it:

  scan           h_t = exp(log_a_t) * h_{t-1} + x_t per channel, over packed sequences (forward, forward and
                 backward as one training step, backward alone, one token per sequence)
  conv           causal depthwise convolution of 2 to 4 taps over packed sequences, with an optional SiLU
                 (forward, backward, one token per sequence)
  norm_gate      RMS norm of every head's output times a gate's activation (forward, backward)
  residual_norm  residual + scale * x and the RMS norm of the sum (forward, backward)

``own`` False: the plain form, elementary torch operations in 32 bits, rounded once at the end.
``own`` True: the calls of this repository's package.
"""
import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ---------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # four sequences answered one token at a time: a call's latency
        dict(name="scan_step_4x2048", op="scan", dir="step", dtype="bf16", tokens=4, seqs=4, channels=2048),
        # one prompt of ordinary length, 16 heads of 128 channels
        dict(name="scan_fwd_1x4096", op="scan", dir="fwd", dtype="bf16", tokens=4096, seqs=1, channels=2048),
        # the long prefill: two sequences of 32K tokens, 32 heads of 128 channels (the largest case)
        dict(name="scan_fwd_2x32768", op="scan", dir="fwd", dtype="bf16", tokens=65536, seqs=2, channels=4096),
        # a training step over a packed batch of ragged sequences in float32, a width that is no power of two
        dict(name="scan_train_ragged", op="scan", dir="train", dtype="f32", tokens=24571, seqs=24, channels=1000),
        # the decode batch: 256 sequences, 32 heads of 128, x a slice of the fused projection
        dict(name="conv_step_256", op="conv", dir="step", dtype="bf16", tokens=256, seqs=256, channels=4096, width=4,
             silu=True, fused=True),
        # a packed prefill of 64 ragged sequences, x a slice of the fused projection
        dict(name="conv_fwd_64seq", op="conv", dir="fwd", dtype="bf16", tokens=65501, seqs=64, channels=4096, width=4,
             silu=True, fused=True),
        # the convolution's gradient in training, two sequences of 16K tokens
        dict(name="conv_bwd_2x16384", op="conv", dir="bwd", dtype="bf16", tokens=32768, seqs=2, channels=4096, width=4,
             silu=True, fused=False),
        # a decode batch's heads: 256 tokens, 32 heads of 128
        dict(name="norm_gate_fwd_256", op="norm_gate", dir="fwd", dtype="bf16", tokens=256, heads=32, width=128,
             act="sigmoid", fused=False),
        # an odd head width and count in float32, the gate a slice of the fused projection
        dict(name="norm_gate_fwd_odd", op="norm_gate", dir="fwd", dtype="f32", tokens=5003, heads=11, width=83,
             act="silu", fused=True),
        # the gradient in training, 32K tokens
        dict(name="norm_gate_bwd_32768", op="norm_gate", dir="bwd", dtype="bf16", tokens=32768, heads=32, width=128,
             act="sigmoid", fused=False),
        # one token through one layer: a call's latency
        dict(name="residual_norm_fwd_1", op="residual_norm", dir="fwd", dtype="bf16", tokens=1, width=4096,
             residual="bf16", channel_scale=False),
        # the gradient in training, a float32 residual stream with a learned scale per channel
        dict(name="residual_norm_bwd_16384", op="residual_norm", dir="bwd", dtype="bf16", tokens=16384, width=4096,
             residual="f32", channel_scale=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan", "conv", "norm_gate", "residual_norm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("scan", "conv"):
        d = rng.choice(["fwd", "train", "bwd", "step"] if op == "scan" else ["fwd", "bwd", "step"])
        channels = _log(rng, 40, 4096)
        if rng.random() < 0.5:
            channels = max(64, channels // 64 * 64)  # whole heads
        if d == "step":
            seqs = _log(rng, 1, 1024)
            tokens = seqs
        else:
            tokens = _log(rng, 1, 65536)
            seqs = _log(rng, 1, min(tokens, 128))
        c = dict(op=op, dir=d, dtype=dtype, tokens=tokens, seqs=seqs, channels=channels)
        if op == "conv":
            c.update(width=rng.choice([2, 3, 4]), silu=rng.random() < 0.7, fused=rng.random() < 0.5)
        return c
    d = rng.choice(["fwd", "bwd"])
    if op == "norm_gate":
        width = rng.choice([16, 32, 64, 128, 256, rng.randint(17, 300)])
        heads = rng.randint(1, 32)
        tokens = _log(rng, 1, min(65536, 134217728 // (heads * width)))
        return dict(op=op, dir=d, dtype=dtype, tokens=tokens, heads=heads, width=width,
                    act=rng.choice(["sigmoid", "silu"]), fused=rng.random() < 0.5)
    width = _log(rng, 200, 8192)
    if rng.random() < 0.6:
        width = max(256, width // 128 * 128)
    tokens = _log(rng, 1, min(65536, 134217728 // width))
    return dict(op=op, dir=d, dtype=dtype, tokens=tokens, width=width,
                residual="f32" if dtype == "f32" else rng.choice(["bf16", "f32"]), channel_scale=rng.random() < 0.5)


def _lengths(c):
    """The sequences' lengths, fixed by the case's sizes alone; equal where they can be (an even batch)."""
    T, N = c["tokens"], c["seqs"]
    if T % N == 0 and N < 8:
        return [T // N] * N
    r = random.Random(1000003 * T + N)
    cuts = sorted(r.randint(0, T) for _ in range(N - 1))  # empty sequences may occur, as in a real batch
    return [b - a for a, b in zip([0] + cuts, cuts + [T])]


def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


# ---------------------------------------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 17)

    def normal(*shape, std=1.0, mean=0.0):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32) * std + mean

    op, d, dt = case["op"], case["dir"], _dt(case["dtype"])
    T = case["tokens"]
    s = {"case": case}
    if op in ("scan", "conv"):
        N, C = case["seqs"], case["channels"]
        if d != "step":
            cu = [0]
            for n in _lengths(case):
                cu.append(cu[-1] + n)
            s["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
    if op == "scan":
        s["x"] = normal(T, C).to(dt)
        # half of the channels forget within tokens, half remember hundreds of them
        fast = -torch.nn.functional.softplus(normal(T, C, std=2.0)).clamp(max=8.0)
        slow = -torch.exp(torch.rand(C, generator=g, device=DEV) * 6.0 - 6.2) * torch.sigmoid(normal(T, C))
        s["log_a"] = torch.where(torch.arange(C, device=DEV) % 2 == 0, fast, slow).contiguous()
        s["h0"] = normal(N, C)
        if d in ("train", "bwd"):
            s["dy"] = normal(T, C).to(dt)
            s["dhT"] = normal(N, C)
    elif op == "conv":
        W = case["width"]
        base = normal(T, 2 * C if case["fused"] else C).to(dt)
        s["x"] = base[:, C:] if case["fused"] else base
        s["weight"] = normal(C, W, std=W ** -0.5)
        s["bias"] = normal(C, std=0.1)
        s["state"] = normal(N, W - 1, C).to(dt)
        if d == "bwd":
            s["dy"] = normal(T, C).to(dt)
            s["dstate_T"] = normal(N, W - 1, C).to(dt)
    elif op == "norm_gate":
        H, D = case["heads"], case["width"]
        s["x"] = (normal(T, H, D) * torch.exp(normal(T, H, 1))).to(dt)
        base = normal(T, 2 * H * D if case["fused"] else H * D, std=1.5).to(dt)
        s["gate"] = (base[:, H * D:] if case["fused"] else base).unflatten(1, (H, D))
        s["weight"] = normal(D, std=0.1, mean=1.0)
        if d == "bwd":
            s["dy"] = normal(T, H, D).to(dt)
    else:
        D = case["width"]
        rt = _dt(case["residual"])
        s["x"] = normal(T, D).to(dt)
        s["res"] = normal(T, D, std=3.0).to(rt)  # the stream before the sum (forward), the sum itself (backward)
        s["weight"] = normal(D, std=0.1, mean=1.0)
        s["scale"] = 0.5
        s["cscale"] = normal(D, std=0.2, mean=0.7) if case["channel_scale"] else None
        if d == "bwd":
            s["dy"] = normal(T, D).to(dt)
            s["dres"] = normal(T, D).to(rt)
    return s


# ---------------------------------------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    op, d = case["op"], case["dir"]
    if own:
        return _OWN[op](s, d)
    return _PLAIN[op](s, d)


def _own_scan(s, d):
    import kda_recurrent_state_amd as kda
    if d == "step":
        y, h = kda.scan_step(s["x"], s["log_a"], s["h0"], h_out=torch.empty_like(s["h0"]))
        return {"y": y, "h": h}
    if d == "fwd":
        y, h = kda.scan_fwd(s["x"], s["log_a"], s["h0"], s["cu"])
        return {"y": y, "h": h}
    out = {}
    states = None
    if d == "train":
        out["y"], out["h"], states = kda.scan_fwd_states(s["x"], s["log_a"], s["h0"], s["cu"])
    out.update(kda.scan_bwd(s["x"], s["log_a"], s["dy"], s["h0"], s["cu"], s["dhT"], states=states))
    return out


def _own_conv(s, d):
    import kda_recurrent_state_amd as kda
    act = "silu" if s["case"]["silu"] else None
    if d == "step":
        y, st = kda.conv_step(s["x"], s["weight"], s["state"], s["bias"], activation=act,
                              state_out=torch.empty_like(s["state"]))
        return {"y": y, "state": st}
    if d == "fwd":
        y, st = kda.conv_fwd(s["x"], s["weight"], s["bias"], s["state"], s["cu"], activation=act)
        return {"y": y, "state": st}
    return kda.conv_bwd(s["x"], s["weight"], s["dy"], s["bias"], s["state"], s["cu"], s["dstate_T"], activation=act)


def _own_norm_gate(s, d):
    import kda_recurrent_state_amd as kda
    act = s["case"]["act"]
    if d == "fwd":
        return kda.norm_gate_fwd(s["x"], s["weight"], s["gate"], activation=act, eps=EPS)
    return kda.norm_gate_bwd(s["x"], s["weight"], s["dy"], s["gate"], activation=act, eps=EPS)


def _own_residual_norm(s, d):
    import kda_recurrent_state_amd as kda
    kw = dict(scale=s["scale"], channel_scale=s["cscale"], eps=EPS)
    if d == "fwd":
        y, r = kda.residual_norm_fwd(s["x"], s["res"], s["weight"], **kw)
        return {"y": y, "residual": r}
    return kda.residual_norm_bwd(s["x"], s["res"], s["weight"], s["dy"], s["dres"], **kw)


_OWN = {"scan": _own_scan, "conv": _own_conv, "norm_gate": _own_norm_gate, "residual_norm": _own_residual_norm}


# ---------------------------------------------------------------------------------------------- plain forms

def _where(cu, T):
    """Sequence of every packed token, and whether it is its sequence's first."""
    t = torch.arange(T, device=cu.device, dtype=torch.int32)
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return seq, t == cu[seq]


def _prefix(a, b):
    """h_t = a_t h_{t-1} + b_t along the first axis from a zero state, by doubling."""
    step = 1
    while step < a.shape[0]:
        b = torch.cat([b[:step], b[step:] + a[step:] * b[:-step]])
        a = torch.cat([a[:step], a[step:] * a[:-step]])
        step *= 2
    return b


def _plain_scan(s, d):
    x, a, h0 = s["x"].float(), torch.exp(s["log_a"]), s["h0"]
    dt = s["x"].dtype
    if d == "step":
        h = a * h0 + x
        return {"y": h.to(dt), "h": h}
    cu = s["cu"]
    T = x.shape[0]
    seq, first = _where(cu, T)
    first = first[:, None]
    start = h0[seq]
    h = _prefix(torch.where(first, 0.0, a), torch.where(first, x + a * start, x))
    empty = (cu[1:] == cu[:-1])[:, None]
    last = (cu[1:].long() - 1).clamp(min=0)
    out = {}
    if d in ("fwd", "train"):
        out["y"], out["h"] = h.to(dt), torch.where(empty, h0, h[last])
    if d in ("train", "bwd"):
        before = torch.where(first, start, torch.cat([h0[:1], h[:-1]]))
        dy, dhT = s["dy"].float(), s["dhT"]
        ends = (torch.arange(T, device=x.device) == cu[1:][seq] - 1)[:, None]
        dy = torch.where(ends, dy + dhT[seq], dy)
        nxt = torch.where(ends, 0.0, torch.cat([a[1:], a[:1]]))  # the factor that carries token t + 1's derivative to t
        dh = _prefix(nxt.flip(0), dy.flip(0)).flip(0)
        begin = cu[:-1].long().clamp(max=T - 1)
        out["dx"], out["dlog_a"] = dh.to(dt), dh * a * before
        out["dh0"] = torch.where(empty, dhT, a[begin] * dh[begin])
    return out


def _plain_conv(s, d):
    x, w, b, state = s["x"].float(), s["weight"], s["bias"], s["state"].float()
    dt, silu = s["x"].dtype, s["case"]["silu"]
    C, W = w.shape
    N = state.shape[0]
    if d == "step":
        full = torch.cat([state, x[:, None]], 1)  # [N, W, C]
        z = (full * w.t()[None]).sum(1) + b
        y = z * torch.sigmoid(z) if silu else z
        return {"y": y.to(dt), "state": full[:, 1:].to(dt)}
    cu = s["cu"]
    T = x.shape[0]
    seq, _ = _where(cu, T)
    # every sequence with its W - 1 earlier inputs in front
    ext = torch.empty(T + N * (W - 1), C, device=x.device)
    at = torch.arange(T, device=x.device) + (seq + 1) * (W - 1)
    front = (cu[:-1].long() + torch.arange(N, device=x.device) * (W - 1))[:, None] + torch.arange(W - 1, device=x.device)
    ext[at] = x
    ext[front.reshape(-1)] = state.reshape(-1, C)
    taps = [ext[at - (W - 1) + j] for j in range(W)]
    z = sum(taps[j] * w[:, j] for j in range(W)) + b
    tail = (cu[1:].long() + torch.arange(N, device=x.device) * (W - 1))[:, None] + torch.arange(W - 1, device=x.device)
    if d == "fwd":
        y = z * torch.sigmoid(z) if silu else z
        return {"y": y.to(dt), "state": ext[tail].to(dt)}
    dz = s["dy"].float()
    if silu:
        sg = torch.sigmoid(z)
        dz = dz * (sg * (1 + z * (1 - sg)))
    dzx = torch.zeros(ext.shape[0] + W - 1, C, device=x.device)
    dzx[at] = dz
    dext = sum(dzx[k:k + ext.shape[0]] * w[:, W - 1 - k] for k in range(W))
    dext.index_add_(0, tail.reshape(-1), s["dstate_T"].float().reshape(-1, C))
    dw = torch.stack([(dz * taps[j]).sum(0, dtype=torch.float64) for j in range(W)], 1).float()
    return {"dx": dext[at].to(dt), "dweight": dw, "dbias": dz.sum(0, dtype=torch.float64).float(),
            "dstate": dext[front].to(dt)}


def _plain_norm_gate(s, d):
    x, w, g = s["x"].float(), s["weight"], s["gate"].float()
    dt = s["x"].dtype
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    sg = torch.sigmoid(g)
    act = g * sg if s["case"]["act"] == "silu" else sg
    if d == "fwd":
        return (x * r * w * act).to(dt)
    dy = s["dy"].float()
    n = x * r
    dn = dy * act * w
    dx = r * (dn - n * (dn * n).mean(-1, keepdim=True))
    slope = sg * (1 + g * (1 - sg)) if s["case"]["act"] == "silu" else sg * (1 - sg)
    dw = (dy * act * n).sum((0, 1), dtype=torch.float64).float()
    return {"dx": dx.to(dt), "dgate": (dy * n * w * slope).to(dt), "dweight": dw}


def _plain_residual_norm(s, d):
    x, res, w = s["x"].float(), s["res"].float(), s["weight"]
    sc = s["scale"] if s["cscale"] is None else s["scale"] * s["cscale"]
    if d == "fwd":
        h = res + sc * x
        y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * w
        return {"y": y.to(s["x"].dtype), "residual": h.to(s["res"].dtype)}
    dy, dres = s["dy"].float(), s["dres"].float()
    r = torch.rsqrt((res * res).mean(-1, keepdim=True) + EPS)
    n = res * r
    dn = dy * w
    dh = dres + r * (dn - n * (dn * n).mean(-1, keepdim=True))
    out = {"dx": (sc * dh).to(s["x"].dtype), "dresidual": dh.to(s["res"].dtype),
           "dweight": (dy * n).sum(0, dtype=torch.float64).float()}
    if s["cscale"] is not None:
        out["dchannel_scale"] = (s["scale"] * dh * x).sum(0, dtype=torch.float64).float()
    return out


_PLAIN = {"scan": _plain_scan, "conv": _plain_conv, "norm_gate": _plain_norm_gate,
          "residual_norm": _plain_residual_norm}


# ---------------------------------------------------------------------------------------------- work

def work(case):
    """Bytes of every input read once and every output written once; operations of the formulas."""
    op, d, T = case["op"], case["dir"], case["tokens"]
    e = 2 if case["dtype"] == "bf16" else 4
    if op == "scan":
        n, st = T * case["channels"], case["seqs"] * case["channels"] * 4
        if d in ("fwd", "step"):
            return {"bytes": n * (2 * e + 4) + 2 * st, "flops": 3 * n}
        return {"bytes": n * (3 * e + 8) + 3 * st + (n * e + st if d == "train" else 0),
                "flops": (8 if d == "train" else 7) * n}
    if op == "conv":
        C, W = case["channels"], case["width"]
        n, st, par = T * C, case["seqs"] * (W - 1) * C * e, C * (W + 1) * 4
        act = 4 * n if case["silu"] else 0
        if d in ("fwd", "step"):
            return {"bytes": n * 2 * e + 2 * st + par, "flops": 2 * W * n + act}
        return {"bytes": n * 3 * e + 3 * st + 2 * par, "flops": (4 * W + (2 * W if case["silu"] else 0) + 1) * n + 2 * act}
    if op == "norm_gate":
        n = T * case["heads"] * case["width"]
        return {"bytes": n * (3 if d == "fwd" else 5) * e + case["width"] * (4 if d == "fwd" else 8),
                "flops": (9 if d == "fwd" else 22) * n}
    D = case["width"]
    n, er, cs = T * D, 2 if case["residual"] == "bf16" else 4, case["channel_scale"]
    if d == "fwd":
        return {"bytes": n * (2 * e + 2 * er) + D * 4 * (2 if cs else 1), "flops": 6 * n}
    return {"bytes": n * (2 * e + 3 * er + (e if cs else 0)) + D * 4 * (4 if cs else 2), "flops": (14 if cs else 11) * n}


# ---------------------------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    """What run() returns, from the operators' definitions in 64 bits: sequence by sequence and token by token for
    the scan and the convolution, gradients by torch's differentiation of the definition (for the scan by its
    recurrence run backwards)."""
    s = prepare(case, seed)
    return {"scan": _exact_scan, "conv": _exact_conv, "norm_gate": _exact_norm_gate,
            "residual_norm": _exact_residual_norm}[case["op"]](s, case)


def _exact_scan(s, case):
    d = case["dir"]
    x, a, h0 = s["x"].double(), s["log_a"].double().exp_(), s["h0"].double()
    if d == "step":
        h = torch.addcmul(x, a, h0)
        return {"y": h, "h": h}
    cu = s["cu"].tolist()
    hs = torch.empty_like(x)
    hT = torch.empty_like(h0)
    for n in range(len(cu) - 1):
        h = h0[n]
        for t in range(cu[n], cu[n + 1]):
            h = torch.addcmul(x[t], a[t], h, out=hs[t])
        hT[n] = h
    out = {"y": hs, "h": hT} if d in ("fwd", "train") else {}
    if d in ("train", "bwd"):
        dy = s["dy"].double()
        dx, dla, dh0 = torch.empty_like(x), torch.empty_like(x), s["dhT"].double()
        for n in range(len(cu) - 1):
            carry = dh0[n].clone()
            for t in reversed(range(cu[n], cu[n + 1])):
                torch.add(dy[t], carry, out=dx[t])
                torch.mul(dx[t], a[t], out=carry)
                torch.mul(carry, hs[t - 1] if t > cu[n] else h0[n], out=dla[t])
            dh0[n] = carry
        out.update(dx=dx, dlog_a=dla, dh0=dh0)
    return out


def _exact_conv(s, case):
    W, d = case["width"], case["dir"]
    grad = d == "bwd"
    x = s["x"].double().requires_grad_(grad)
    w, b = (s[k].double().requires_grad_(grad) for k in ("weight", "bias"))
    state = s["state"].double().requires_grad_(grad)
    cu = list(range(case["seqs"] + 1)) if d == "step" else s["cu"].tolist()
    ys, sts = [], []
    for n in range(len(cu) - 1):
        L = cu[n + 1] - cu[n]
        seq = torch.cat([state[n], x[cu[n]:cu[n + 1]]])
        z = b.expand(L, -1)
        for j in range(W):
            z = z + w[:, j] * seq[j:j + L]
        ys.append(z / (1 + torch.exp(-z)) if case["silu"] else z)
        sts.append(seq[L:])
    y, st = torch.cat(ys), torch.stack(sts)
    if not grad:
        return {"y": y, "state": st}
    dx, dw, db, ds = torch.autograd.grad([y, st], [x, w, b, state], [s["dy"].double(), s["dstate_T"].double()])
    return {"dx": dx, "dweight": dw, "dbias": db, "dstate": ds}


def _exact_norm_gate(s, case):
    grad = case["dir"] == "bwd"
    x, w, g = (s[k].double().requires_grad_(grad) for k in ("x", "weight", "gate"))
    act = 1 / (1 + torch.exp(-g))
    if case["act"] == "silu":
        act = g * act
    y = x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS) * w * act
    if not grad:
        return y.detach()
    dx, dw, dg = torch.autograd.grad(y, [x, w, g], s["dy"].double())
    return {"dx": dx, "dgate": dg, "dweight": dw}


def _exact_residual_norm(s, case):
    def norm(h, w):
        return h / torch.sqrt(h.square().sum(-1, keepdim=True) / h.shape[-1] + EPS) * w

    x, res, w = s["x"].double(), s["res"].double(), s["weight"].double()
    sc = s["scale"] * (s["cscale"].double() if s["cscale"] is not None else 1.0)
    if case["dir"] == "fwd":
        h = res + sc * x
        return {"y": norm(h, w), "residual": h}
    # backward at the given sum: what reaches the sum from both sides, then its two addends and the scale
    h, w = res.requires_grad_(True), w.requires_grad_(True)
    dh, dw = torch.autograd.grad(norm(h, w), [h, w], s["dy"].double())
    dh = dh + s["dres"].double()
    out = {"dx": sc * dh, "dresidual": dh, "dweight": dw}
    if s["cscale"] is not None:
        out["dchannel_scale"] = (s["scale"] * dh * x).sum(0)
    return out
