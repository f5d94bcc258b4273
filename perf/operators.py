"""Cases of the selective state space block's operators, for timing and for comparing outputs.

Three operators: the short causal convolution with its bias, activation and carried rows ("conv"), the
selective state space scan ("scan") and the matrix product with bias, activation and residual in its
epilogue ("linear"), which are the block's parts in the order in which its data pass them. A case
says which operator, which of its forms (a prompt, a training step with its gradients, a single
token) and the sizes. Where ``own`` is false ``run`` computes the plain form in 32 bits; where it is
true it calls this repository's entry points.

  conv    y[t] = act(bias + sum_k weight[k] x[t-W+1+k]), rows before the first from the carried state
  scan    d = softplus(dt + dt_bias); h[t] = exp(d A) h[t-1] + d B[t] x[t];
          out[t] = (sum_n C[t,n] h[t,n] + D x[t]) * silu(z[t])
  linear  out = act(x weight^T + bias) + residual

Rows at or past a sequence's length give zeros and leave its state alone.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
DEVICE = "cuda"


def _mdc():
    import masked_depthwise_causal_amd

    return masked_depthwise_causal_amd


# -- cases -------------------------------------------------------------------------------------------
def _conv(name, form, dtype, S, B, H, W, ragged=False):
    return {"name": name, "op": "conv", "form": form, "dtype": dtype, "S": S, "B": B, "H": H, "W": W,
            "ragged": ragged}


def _scan(name, form, dtype, S, B, H, N, G=1, ragged=False, gate=True):
    return {"name": name, "op": "scan", "form": form, "dtype": dtype, "S": S, "B": B, "H": H, "N": N,
            "G": G, "ragged": ragged, "gate": gate}


def _linear(name, form, dtype, M, K, N, act, residual=False, extra=0):
    return {"name": name, "op": "linear", "form": form, "dtype": dtype, "M": M, "K": K, "N": N,
            "act": act, "residual": residual, "extra": extra}


def listed():
    return [
        # one token of eight sequences in a serving loop: a call of some 0.4 MB, where latency counts
        _conv("conv_token", "step", "bf16", 1, 8, 5120, 4),
        # prompts of unequal, odd lengths that continue earlier ones, channels no power of two
        _conv("conv_prompt_ragged", "prompt", "fp16", 1537, 5, 1000, 3, ragged=True),
        # a training step; x is the one half of the block's first projection, so its rows are strided
        _conv("conv_train", "train", "bf16", 4096, 4, 4096, 4),
        # one token of 64 sequences: the state is read and written once
        _scan("scan_token", "step", "bf16", 1, 64, 5120, 16),
        # one long prompt, with few channels for the card: the work has to be split over its length
        _scan("scan_prompt_long", "prompt", "bf16", 16384, 1, 4096, 16),
        # ragged prompts, two groups of B and C, a small state, no gate, odd sizes
        _scan("scan_prompt_ragged", "prompt", "fp16", 777, 5, 1000, 8, G=2, ragged=True, gate=False),
        # a training step's forward and backward at an ordinary size
        _scan("scan_train", "train", "bf16", 2048, 8, 4096, 16),
        # a training step of a small model, ragged
        _scan("scan_train_small", "train", "fp16", 513, 2, 384, 16, ragged=True),
        # the block's last projection for one token of four sequences: the weight is read once
        _linear("linear_token", "forward", "bf16", 4, 5120, 4096, "none", residual=True),
        # a step size's projection of odd rank, read out of wider rows, with its softplus
        _linear("linear_rank_odd", "forward", "fp16", 3885, 63, 1000, "softplus", extra=32),
        # the block's first projection over a prompt
        _linear("linear_prompt", "forward", "bf16", 4096, 4096, 8192, "silu"),
        # a projection's training step: product, activation and residual, and their gradients
        _linear("linear_train", "train", "bf16", 4096, 5120, 4096, "silu", residual=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _channels(rng, lo, hi, multiple):
    """A channel count spread over its logarithm: a multiple of 64 three times of four, else odd ones."""
    h = _log_int(rng, lo, hi)
    m = multiple * (64 if rng.random() < 0.75 else 1)
    return max(m, h // m * m)


def draw(rng):
    op = rng.choice(("conv", "scan", "linear"))
    dtype = rng.choice(("bf16", "fp16"))
    ragged = rng.random() < 0.4
    if op == "linear":
        form = rng.choice(("forward", "forward", "train"))
        most = 4096 * 4096 * 8192 // (3 if form == "train" else 1)
        N, K = _log_int(rng, 64, 8192), _log_int(rng, 32, 8192)
        if rng.random() < 0.6:
            N, K = max(64, N // 64 * 64), max(32, K // 32 * 32)
        M = _log_int(rng, 1, max(1, min(8192, most // (N * K))))
        act = rng.choice(("none", "relu", "silu", "gelu", "softplus"))
        c = _linear("", form, dtype, M, K, N, act, rng.random() < 0.5, rng.choice((0, 0, 8, 33)))
    else:
        form = rng.choice(("prompt", "train", "step"))
        B = _log_int(rng, 1, 64 if form == "step" else 16)
        G = rng.choice((1, 1, 2, 4)) if op == "scan" else 1
        H = _channels(rng, 64, 8192, G)
        N = rng.choice((1, 4, 7, 8, 16, 16, 16, 24, 32)) if op == "scan" else 1
        most = 2 ** 26 if op == "conv" else 2 ** 30
        S = 1 if form == "step" else _log_int(rng, 1, max(1, min(16384, most // (B * H * N))))
        if op == "conv":
            c = _conv("", form, dtype, S, B, H, rng.choice((2, 3, 4, 4)), ragged and form != "step")
        else:
            c = _scan("", form, dtype, S, B, H, N, G, ragged and form != "step", rng.random() < 0.7)
    del c["name"]
    return c


# -- inputs ------------------------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed * 1009 + 17)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return torch.randn(shape, generator=g, device=DEVICE).mul_(scale).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(shape, generator=g, device=DEVICE).mul_(hi - lo).add_(lo)

    s = {"case": case}
    if case["op"] == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        s["x"] = normal(M, K + case["extra"])[:, :K]  # a part of wider rows where extra > 0
        s["weight"] = normal(N, K, scale=K ** -0.5)
        s["bias"] = normal(N, scale=0.5)
        s["residual"] = normal(M, N) if case["residual"] else None
        if case["form"] == "train":
            s["gout"] = normal(M, N)
        return s
    S, B, H = case["S"], case["B"], case["H"]
    train, step = case["form"] == "train", case["form"] == "step"
    s["lengths"] = None
    if case["ragged"]:
        s["lengths"] = torch.randint(0, S + 1, (B,), generator=g, device=DEVICE)
        s["lengths"][0] = S  # the longest gives the padded size
    if case["op"] == "conv":
        W = case["W"]
        s["x"] = normal(B, H) if step else normal(S, B, 2 * H)[:, :, :H]
        s["weight"], s["bias"] = normal(W, H, scale=0.5), normal(H, scale=0.5)
        s["state"] = None if train else normal(W - 1, B, H)
        if train:
            s["gout"] = normal(S, B, H)
        return s
    N, G = case["N"], case["G"]
    rows = (B,) if step else (S, B)
    # x as the convolution's activation leaves it; B and C are parts of one projection's rows
    x = normal(*rows, H, dtype=torch.float32)
    s["x"] = (x * torch.sigmoid(x)).to(dt)
    s["dt"] = normal(*rows, H, scale=0.5)
    bc = normal(*rows, G, 2 * N)
    s["B"], s["C"] = bc[..., :N], bc[..., N:]
    s["z"] = normal(*rows, H) if case["gate"] else None
    # decay rates near 1..N and step sizes between 1e-3 and 0.1, the usual start of training
    rate = torch.arange(1, N + 1, device=DEVICE, dtype=torch.float32)[:, None]
    s["A"] = -rate * torch.exp(normal(N, H, scale=0.2, dtype=torch.float32))
    s["D"] = 1 + normal(H, scale=0.1, dtype=torch.float32)
    d = torch.exp(uniform(H, lo=math.log(1e-3), hi=math.log(0.1)))
    s["dt_bias"] = torch.log(torch.expm1(d))
    s["state"] = None if train else normal(B, N, H, dtype=torch.float32)
    if train:
        s["gout"] = normal(*rows, H)
    return s


# -- the plain form ----------------------------------------------------------------------------------
def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-torch.abs(v)))


def _act(v, act):
    if act == "relu":
        return torch.clamp(v, min=0)
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return _softplus(v) if act == "softplus" else v


def _act_slope(v, act):
    if act == "relu":
        return (v > 0).to(v.dtype)
    if act == "silu":
        g = torch.sigmoid(v)
        return g * (1 + v * (1 - g))
    if act == "gelu":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (v + 0.044715 * v * v * v))
        return 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * c * (1 + 3 * 0.044715 * v * v)
    return torch.sigmoid(v) if act == "softplus" else torch.ones_like(v)


def _live(S, B, lengths):
    """[S,B,1]: whether a row is before its sequence's length."""
    if lengths is None:
        return torch.ones((S, B, 1), dtype=torch.bool, device=DEVICE)
    return (torch.arange(S, device=DEVICE)[:, None] < lengths[None, :])[:, :, None]


def _shift(v, k, S):
    """v's rows k..k+S-1, for v of at least S + k rows."""
    return v[k:k + S]


def _plain_conv(s):
    c = s["case"]
    W, B, H = c["W"], c["B"], c["H"]
    dt, w, bias = s["x"].dtype, s["weight"].float(), s["bias"].float()
    if c["form"] == "step":
        rows = torch.cat([s["state"], s["x"][None]])
        y = _act((rows.float() * w[:, None]).sum(0) + bias, "silu")
        s["state"].copy_(rows[1:].clone())
        return {"y": y.to(dt), "state": s["state"]}
    S = c["S"]
    live = _live(S, B, s["lengths"])
    x = torch.where(live, s["x"].float(), 0.0)
    before = torch.zeros((W - 1, B, H), device=DEVICE) if s["state"] is None else s["state"].float()
    rows = torch.cat([before, x])
    pre = sum(w[k] * _shift(rows, k, S) for k in range(W)) + bias
    y = torch.where(live, _act(pre, "silu"), 0.0)
    if c["form"] == "prompt":
        length = torch.full((B,), S, device=DEVICE) if s["lengths"] is None else s["lengths"]
        at = torch.arange(W - 1, device=DEVICE)[:, None] + length[None, :]  # in rows
        state = rows.gather(0, at[:, :, None].expand(W - 1, B, H))
        return {"y": y.to(dt), "state": state.to(dt)}
    gpre = torch.where(live, s["gout"].float() * _act_slope(pre, "silu"), 0.0)
    after = torch.cat([gpre, torch.zeros((W - 1, B, H), device=DEVICE)])
    gx = torch.where(live, sum(w[W - 1 - k] * _shift(after, k, S) for k in range(W)), 0.0)
    gw = torch.stack([(gpre * _shift(rows, k, S)).sum((0, 1)) for k in range(W)])
    return {"y": y.to(dt), "gx": gx.to(dt), "gw": gw.to(dt), "gbias": gpre.sum((0, 1)).to(dt)}


def _recur(a, b, reverse=False):
    """h[t] = a[t] h[t-1] + b[t] for all t, or h[t] = a[t+1] h[t+1] + b[t], by doubling the span."""
    S, k = a.shape[0], 1
    if reverse:
        a = torch.cat([a[1:], torch.ones_like(a[:1])])
    while k < S:
        nb, na = b.clone(), a.clone()
        if reverse:
            nb[:-k].addcmul_(a[:-k], b[k:])
            na[:-k].mul_(a[k:])
        else:
            nb[k:].addcmul_(a[k:], b[:-k])
            na[k:].mul_(a[:-k])
        a, b, k = na, nb, 2 * k
    return b


def _plain_scan(s):
    c = s["case"]
    B, H, N, G = c["B"], c["H"], c["N"], c["G"]
    K, dt = H // G, s["x"].dtype
    A = s["A"].view(N, G, K)
    if c["form"] == "step":
        d = _softplus(s["dt"].float() + s["dt_bias"]).view(B, 1, G, K)
        x = s["x"].float().view(B, 1, G, K)
        Bm, Cm = (s[n].float().transpose(1, 2)[..., None] for n in ("B", "C"))
        h = torch.exp(d * A) * s["state"].view(B, N, G, K) + d * x * Bm
        y = (h * Cm).sum(1) + s["D"].view(G, K) * x[:, 0]
        s["state"].copy_(h.view(B, N, H))
        y = y.view(B, H)
        y = y if s["z"] is None else y * _act(s["z"].float(), "silu")
        return {"out": y.to(dt), "state": s["state"]}
    S = c["S"]
    live = _live(S, B, s["lengths"])
    x = torch.where(live, s["x"].float(), 0.0)
    raw = s["dt"].float() + s["dt_bias"]
    d = torch.where(live, _softplus(raw), 0.0)
    # [S,B,N,G,K] throughout: states outside channels, channels in their groups
    Bm, Cm = (torch.where(live[..., None], s[n].float(), 0.0).transpose(2, 3)[..., None]
              for n in ("B", "C"))
    D4, x4 = d.view(S, B, 1, G, K), x.view(S, B, 1, G, K)
    a = torch.exp(D4 * A)
    b = (D4 * x4) * Bm
    if s["state"] is not None:
        b[0] += a[0] * s["state"].view(B, N, G, K)
    h = _recur(a, b)
    y = (h * Cm).sum(2).view(S, B, H) + s["D"] * x
    gate = None if s["z"] is None else torch.where(live, s["z"].float(), 0.0)
    out = y if gate is None else y * _act(gate, "silu")
    out = torch.where(live, out, 0.0).to(dt)
    if c["form"] == "prompt":
        return {"out": out, "state": h[-1].reshape(B, N, H)}
    del b
    gout = torch.where(live, s["gout"].float(), 0.0)
    gy = gout if gate is None else gout * _act(gate, "silu")
    gh = _recur(a, gy.view(S, B, 1, G, K) * Cm, reverse=True)
    gB = (gh * (D4 * x4)).sum(4).transpose(2, 3)
    gC = (h * gy.view(S, B, 1, G, K)).sum(4).transpose(2, 3)
    into_u = (gh * Bm).sum(2).view(S, B, H)  # the gradient of d x
    h = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    ga = gh.mul_(h).mul_(a)  # the gradient of d A
    del h, a
    gA = (ga * D4).sum((0, 1)).view(N, H)
    gd = ga.mul_(A).sum(2).view(S, B, H) + into_u * x
    graw = torch.where(live, gd * torch.sigmoid(raw), 0.0)
    got = {"out": out, "gx": torch.where(live, into_u * d + s["D"] * gy, 0.0).to(dt),
           "gdt": graw.to(dt), "gA": gA, "gB": gB.to(dt), "gC": gC.to(dt),
           "gD": (gy * x).sum((0, 1)), "gdt_bias": graw.sum((0, 1))}
    if gate is not None:
        got["gz"] = (gout * y * _act_slope(gate, "silu")).to(dt)
    return got


def _plain_linear(s):
    c = s["case"]
    dt, x, w = s["x"].dtype, s["x"].float(), s["weight"].float()
    pre = x @ w.t() + s["bias"].float()
    out = _act(pre, c["act"])
    if s["residual"] is not None:
        out = out + s["residual"].float()
    if c["form"] == "forward":
        return {"out": out.to(dt)}
    g = s["gout"].float() * _act_slope(pre, c["act"])
    return {"out": out.to(dt), "gx": (g @ w).to(dt), "gw": (g.t() @ x).to(dt),
            "gbias": g.sum(0).to(dt)}


# -- the framework's calls ---------------------------------------------------------------------------
def _own_conv(s):
    mdc, form = _mdc(), s["case"]["form"]
    if form == "step":
        y = mdc.conv_act_step(s["x"], s["weight"], s["state"], s["bias"], activation="silu")
        return {"y": y, "state": s["state"]}
    if form == "prompt":
        y, state = mdc.conv_act_forward(s["x"], s["weight"], s["bias"], activation="silu",
                                        lengths=s["lengths"], state=s["state"], return_state=True)
        return {"y": y, "state": state}
    y = mdc.conv_act_forward(s["x"], s["weight"], s["bias"], activation="silu",
                             lengths=s["lengths"])
    g = mdc.conv_act_backward(s["gout"], s["x"], s["weight"], s["bias"], activation="silu",
                              lengths=s["lengths"])
    return {"y": y, "gx": g.x, "gw": g.weight, "gbias": g.bias}


def _own_scan(s):
    mdc, form = _mdc(), s["case"]["form"]
    if form == "step":
        out = mdc.scan_step(s["state"], s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"],
                            z=s["z"], dt_bias=s["dt_bias"])
        return {"out": out, "state": s["state"]}
    args = {"D": s["D"], "z": s["z"], "dt_bias": s["dt_bias"], "lengths": s["lengths"]}
    ins = (s["x"], s["dt"], s["A"], s["B"], s["C"])
    if form == "prompt":
        out, state = mdc.scan_forward(*ins, **args, state=s["state"], return_state=True)
        return {"out": out, "state": state}
    out, saved = mdc.scan_forward(*ins, **args, return_saved=True)
    g = mdc.scan_backward(s["gout"], *ins, saved, **args)
    got = {"out": out, "gx": g.x, "gdt": g.dt, "gA": g.A, "gB": g.B, "gC": g.C, "gD": g.D,
           "gdt_bias": g.dt_bias}
    if s["z"] is not None:
        got["gz"] = g.z
    return got


def _own_linear(s):
    mdc, c = _mdc(), s["case"]
    act = None if c["act"] == "none" else c["act"]
    if c["form"] == "forward":
        return {"out": mdc.linear_forward(s["x"], s["weight"], s["bias"], activation=act,
                                          residual=s["residual"])}
    out, pre = mdc.linear_forward(s["x"], s["weight"], s["bias"], activation=act,
                                  residual=s["residual"], return_pre=True)
    g = mdc.linear_backward(s["gout"], s["x"], s["weight"], pre, activation=act)
    return {"out": out, "gx": g.x, "gw": g.weight, "gbias": g.bias}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"conv": _own_conv, "scan": _own_scan, "linear": _own_linear}[op](state)
    return {"conv": _plain_conv, "scan": _plain_scan, "linear": _plain_linear}[op](state)


# -- what a pass cannot do without -------------------------------------------------------------------
def work(case):
    """Bytes: every input once, every output once. A training step counts its forward and its
    backward, each with the inputs that it reads. Operations: a product and a sum are two, an
    exponential one. Ragged lengths are uniform, so half of the rows count on average."""
    if case["op"] == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        x, w, out = 2 * M * K, 2 * N * K, 2 * M * N
        fwd = x + w + 2 * N + out * (2 if case["residual"] else 1)
        if case["form"] == "forward":
            return {"bytes": fwd, "flops": 2 * M * K * N}
        return {"bytes": fwd + 2 * (x + w) + out + 2 * N, "flops": 6 * M * K * N}
    S, B, H = case["S"], case["B"], case["H"]
    rows = B if case["form"] == "step" else S * B
    live = rows / 2 if case["ragged"] else rows
    n, part = 2 * rows * H, 2 * live * H  # what is written whole, and what only live rows need
    if case["op"] == "conv":
        W = case["W"]
        weights, state = 2 * (W + 1) * H, 2 * (W - 1) * B * H
        ops = live * H * (2 * W + 4)
        if case["form"] == "train":
            return {"bytes": part + n + 2 * part + n + 2 * weights, "flops": 3 * ops}
        return {"bytes": part + n + weights + 2 * state, "flops": ops}
    N, G = case["N"], case["G"]
    bc, params, state = 4 * live * G * N, 4 * H * (N + 2), 4 * B * N * H
    ins = part * (3 if case["gate"] else 2) + bc + params
    ops = live * H * N
    if case["form"] == "train":
        grads = n * (3 if case["gate"] else 2) + 4 * rows * G * N + params
        return {"bytes": ins + n + ins + part + grads, "flops": 7 * ops + 22 * ops}
    return {"bytes": ins + n + 2 * state, "flops": 7 * ops}


# -- the definition in 64 bits -----------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": _exact_conv, "scan": _exact_scan, "linear": _exact_linear}[case["op"]](case, s)


def _silu64(v):
    return v / (1 + torch.exp(-v))


def _silu64_slope(v):
    e = torch.exp(-v)
    return (1 + e + v * e) / (1 + e) ** 2


def _exact_conv(case, s):
    """Row by row with a window of the last W rows, each sequence's end by comparing row numbers."""
    W, S, B, H = case["W"], case["S"], case["B"], case["H"]
    f = torch.float64
    w, bias = s["weight"].to(f), s["bias"].to(f)
    x = (s["x"][None] if case["form"] == "step" else s["x"]).to(f)
    last = torch.full((B,), S, device=DEVICE) if s["lengths"] is None else s["lengths"]
    window = [torch.zeros((B, H), dtype=f, device=DEVICE) for _ in range(W - 1)]
    if s["state"] is not None:
        window = list(s["state"].to(f))
    y = torch.zeros((S, B, H), dtype=f, device=DEVICE)
    train = case["form"] == "train"
    gx = torch.zeros_like(y) if train else None
    gw, gb = torch.zeros((W, H), dtype=f, device=DEVICE), torch.zeros(H, dtype=f, device=DEVICE)
    for t in range(S):
        on = (t < last)[:, None]
        taps = window + [x[t]]
        pre = bias.expand(B, H).clone()
        for k in range(W):
            pre += w[k] * taps[k]
        y[t] = torch.where(on, _silu64(pre), 0.0)
        if train:
            g = torch.where(on, s["gout"][t].to(f) * _silu64_slope(pre), 0.0)
            gb += g.sum(0)
            for k in range(W):
                gw[k] += torch.where(on, g * taps[k], 0.0).sum(0)
                if t - W + 1 + k >= 0:
                    gx[t - W + 1 + k] += w[k] * g
        window = [torch.where(on, new, old) for new, old in zip(taps[1:], taps[:-1])]
    if train:
        return {"y": y, "gx": gx, "gw": gw, "gbias": gb}
    state = torch.stack(window) if window else torch.zeros((0, B, H), dtype=f, device=DEVICE)
    return {"y": y[0] if case["form"] == "step" else y, "state": state}


def _exact_scan(case, s):
    """One row after the other, as the recurrence is written; the backward by walking back over the
    kept states."""
    S, B, H, N, G = case["S"], case["B"], case["H"], case["N"], case["G"]
    f, step, train = torch.float64, case["form"] == "step", case["form"] == "train"
    row = (lambda n: s[n][None]) if step else (lambda n: s[n])
    X, DT, Bs, Cs = row("x"), row("dt"), row("B"), row("C")
    Z = None if s["z"] is None else row("z")
    A, D, bias = s["A"].to(f), s["D"].to(f), s["dt_bias"].to(f)
    group = torch.arange(H, device=DEVICE) // (H // G)
    last = torch.full((B,), S, device=DEVICE) if s["lengths"] is None else s["lengths"]
    h = torch.zeros((B, N, H), dtype=f, device=DEVICE) if s["state"] is None else s["state"].to(f)
    out = torch.zeros((S, B, H), dtype=f, device=DEVICE)
    kept = torch.zeros((S + 1, B, N, H), dtype=f, device=DEVICE) if train else None
    spread = lambda v: v.to(f).index_select(1, group).transpose(1, 2)  # noqa: E731  [B,G,N] -> [B,N,H]
    for t in range(S):
        on = (t < last)[:, None]
        d = torch.logaddexp(DT[t].to(f) + bias, torch.zeros((), dtype=f, device=DEVICE))
        x = X[t].to(f)
        new = torch.exp(d[:, None] * A) * h + (d * x)[:, None] * spread(Bs[t])
        h = torch.where(on[:, None], new, h)
        y = (spread(Cs[t]) * h).sum(1) + D * x
        if Z is not None:
            y = y * _silu64(Z[t].to(f))
        out[t] = torch.where(on, y, 0.0)
        if train:
            kept[t + 1] = h
    if not train:
        return {"out": out[0] if step else out, "state": h}
    zero = lambda *shape: torch.zeros(shape, dtype=f, device=DEVICE)  # noqa: E731
    got = {"out": out, "gx": zero(S, B, H), "gdt": zero(S, B, H), "gA": zero(N, H),
           "gB": zero(S, B, G, N), "gC": zero(S, B, G, N), "gD": zero(H), "gdt_bias": zero(H)}
    if Z is not None:
        got["gz"] = zero(S, B, H)
    gh = zero(B, N, H)
    for t in range(S - 1, -1, -1):
        on = (t < last)[:, None]
        v, x = DT[t].to(f) + bias, X[t].to(f)
        d = torch.logaddexp(v, torch.zeros((), dtype=f, device=DEVICE))
        Bt, Ct, go = spread(Bs[t]), spread(Cs[t]), torch.where(on, s["gout"][t].to(f), 0.0)
        y = (Ct * kept[t + 1]).sum(1) + D * x
        if Z is not None:
            z = Z[t].to(f)
            got["gz"][t] = go * y * _silu64_slope(z)
            go = go * _silu64(z)
        g = gh + go[:, None] * Ct  # the gradient of h[t]
        got["gC"][t] = (go[:, None] * kept[t + 1]).view(B, N, G, H // G).sum(3).transpose(1, 2)
        got["gB"][t] = torch.where(on[:, None], (g * (d * x)[:, None]).view(B, N, G, H // G).sum(3)
                                   .transpose(1, 2), 0.0)
        a = torch.exp(d[:, None] * A)
        through = (g * Bt).sum(1)
        got["gx"][t] = torch.where(on, through * d + D * go, 0.0)
        ga = torch.where(on[:, None], g * kept[t] * a, 0.0)
        got["gA"] += (ga * d[:, None]).sum(0)
        gv = torch.where(on, ((ga * A).sum(1) + through * x) / (1 + torch.exp(-v)), 0.0)
        got["gdt"][t] = gv
        got["gdt_bias"] += gv.sum(0)
        got["gD"] += (go * x).sum(0)
        gh = torch.where(on[:, None], g * a, gh)
    return got


def _exact_linear(case, s):
    f = torch.float64
    x, w = s["x"].to(f), s["weight"].to(f)
    pre = torch.addmm(s["bias"].to(f), x, w.t())
    one, zero = torch.ones((), dtype=f, device=DEVICE), torch.zeros((), dtype=f, device=DEVICE)
    if case["act"] == "relu":
        out, slope = torch.maximum(pre, zero), torch.where(pre > 0, one, zero)
    elif case["act"] == "silu":
        out, slope = _silu64(pre), _silu64_slope(pre)
    elif case["act"] == "softplus":
        out, slope = torch.logaddexp(pre, zero), 1 / (1 + torch.exp(-pre))
    elif case["act"] == "gelu":  # 0.5 (1 + tanh u) is the logistic function of 2 u
        u = math.sqrt(8 / math.pi) * (pre + 0.044715 * pre ** 3)
        q = 1 / (1 + torch.exp(-u))
        out = pre * q
        slope = q + pre * q * (1 - q) * math.sqrt(8 / math.pi) * (1 + 0.134145 * pre ** 2)
    else:
        out, slope = pre, torch.ones_like(pre)
    if s["residual"] is not None:
        out = out + s["residual"].to(f)
    if case["form"] == "forward":
        return {"out": out}
    g = s["gout"].to(f) * slope
    return {"out": out, "gx": g @ w, "gw": g.t() @ x, "gbias": g.sum(0)}
