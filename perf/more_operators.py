"""Cases of the gated delta rule and of the norms around a block, for timing and for comparing outputs.

Three operators: the gated delta rule ("delta"), which takes the selective scan's place in a block, the
norm before a block with the scaled residual addition ("prenorm") and the norm after a block with its
gate, residual scale and addition ("postnorm"). A case says which operator, which of its forms (a
prompt, a training step with its gradients, a single token) and the sizes. Where ``own`` is false
``run`` computes the plain form in 32 bits; where it is true it calls this repository's entry points.

  delta     d = softplus(dt + dt_bias), a = exp(A d), beta = sigmoid(b), kn = k / |k|, qn = scale q / |q|;
            u = beta (v - a S^T kn), S <- a S + kn u^T, out = S^T qn
  prenorm   r = residual + scale x, out = r / sqrt(mean(r^2) + eps) * weight
  postnorm  out = residual + scale (x / sqrt(mean(x^2 over a group) + eps) * weight * silu(z))

Rows at or past a sequence's length give zeros and leave its state alone.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
DEVICE = "cuda"
EPS = 1e-6  # in |k|^2 + EPS and in the norms' means


def _mdc():
    import masked_depthwise_causal_amd

    return masked_depthwise_causal_amd


# -- cases -------------------------------------------------------------------------------------------
def _delta(name, form, dtype, S, B, H, G, K, V, ragged=False, normalize=True, carry=False):
    return {"name": name, "op": "delta", "form": form, "dtype": dtype, "S": S, "B": B, "H": H, "G": G,
            "K": K, "V": V, "ragged": ragged, "normalize": normalize, "carry": carry}


def _prenorm(name, form, dtype, R, H, scale=True, residual=True, extra=0):
    return {"name": name, "op": "prenorm", "form": form, "dtype": dtype, "R": R, "H": H, "scale": scale,
            "residual": residual, "extra": extra}


def _postnorm(name, form, dtype, R, H, groups, shared=False, gate=True, residual=True, scale=True,
              extra=0):
    return {"name": name, "op": "postnorm", "form": form, "dtype": dtype, "R": R, "H": H,
            "groups": groups, "shared": shared, "gate": gate, "residual": residual, "scale": scale,
            "extra": extra}


def listed():
    return [
        # one token of 32 sequences in a serving loop: the state is read and written once
        _delta("delta_token", "step", "bf16", 1, 32, 16, 16, 128, 128),
        # one token of one sequence of a small model, where latency counts
        _delta("delta_token_small", "step", "fp16", 1, 1, 6, 3, 64, 64),
        # prompts of four sequences, two value heads to a key head
        _delta("delta_prompt", "prompt", "bf16", 4096, 4, 32, 16, 128, 128),
        # one long prompt with few heads for the card
        _delta("delta_prompt_long", "prompt", "bf16", 16384, 1, 16, 16, 128, 128),
        # ragged prompts, odd sizes, keys that come normalized already
        _delta("delta_prompt_ragged", "prompt", "fp16", 777, 5, 6, 2, 96, 80, ragged=True,
               normalize=False),
        # a training step's forward and backward at an ordinary size
        _delta("delta_train", "train", "bf16", 2048, 4, 16, 16, 128, 128),
        # a training step of a small model, ragged, shared keys, from a carried state
        _delta("delta_train_small", "train", "fp16", 513, 2, 6, 3, 64, 128, ragged=True, carry=True),
        # the norm before a block for one token of eight sequences
        _prenorm("prenorm_token", "forward", "bf16", 8, 4096),
        # the same in a training step: the addition, the norm and their gradients
        _prenorm("prenorm_train", "train", "bf16", 16384, 4096),
        # the norm between mixer and last projection over a prompt, a group for each head, one weight for all
        _postnorm("postnorm_prompt", "forward", "bf16", 16384, 4096, 32, shared=True, residual=False,
                  scale=False),
        # the norm after a block, its gate and its addition in a training step
        _postnorm("postnorm_train", "train", "bf16", 16384, 5120, 1),
        # a training step with odd groups, out of wider rows
        _postnorm("postnorm_train_odd", "train", "fp16", 3885, 1000, 8, residual=False, scale=False,
                  extra=33),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("delta", "delta", "prenorm", "postnorm"))
    dtype = rng.choice(("bf16", "fp16"))
    if op == "delta":
        form = rng.choice(("prompt", "train", "step"))
        K = rng.choice((64, 128, 128, _log_int(rng, 8, 128)))
        V = rng.choice((64, 128, 128, _log_int(rng, 8, 256)))
        G = _log_int(rng, 1, 16)
        H = G * rng.choice((1, 1, 2, 4))
        B = _log_int(rng, 1, 32 if form == "step" else 8)
        most = 2 ** 32 if form == "prompt" else 2 ** 31
        S = 1 if form == "step" else _log_int(rng, 1, max(1, min(16384, most // (B * H * K * V))))
        c = _delta("", form, dtype, S, B, H, G, K, V, rng.random() < 0.4 and form != "step",
                   rng.random() < 0.7, rng.random() < 0.5 and form == "train")
    else:
        form = rng.choice(("forward", "train"))
        H = _log_int(rng, 64, 16384)
        if rng.random() < 0.7:
            H = max(64, H // 64 * 64)
        R = _log_int(rng, 1, max(1, min(65536, 2 ** 26 // H)))
        extra = rng.choice((0, 0, 8, 33))
        if op == "prenorm":
            c = _prenorm("", form, dtype, R, H, rng.random() < 0.6, rng.random() < 0.8, extra)
        else:
            groups = rng.choice([1, 1] + [n for n in (2, 4, 5, 8, 16, 32, 64) if H % n == 0])
            c = _postnorm("", form, dtype, R, H, groups, groups > 1 and rng.random() < 0.5,
                          rng.random() < 0.7, rng.random() < 0.5, rng.random() < 0.5, extra)
    del c["name"]
    return c


# -- inputs ------------------------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed * 1013 + 29)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return torch.randn(shape, generator=g, device=DEVICE).mul_(scale).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(shape, generator=g, device=DEVICE).mul_(hi - lo).add_(lo)

    s = {"case": case}
    if case["op"] != "delta":
        R, H, extra = case["R"], case["H"], case["extra"]
        s["x"] = normal(R, H + extra)[:, :H]  # a part of wider rows where extra > 0
        n = H // case["groups"] if case.get("shared") else H
        s["weight"] = (1 + normal(n, scale=0.2, dtype=torch.float32)).to(dt)
        s["residual"] = normal(R, H, scale=2.0) if case["residual"] else None
        s["scale"] = uniform(H, lo=0.1, hi=1.0).to(dt) if case["scale"] else None
        s["z"] = normal(R, H + extra)[:, :H] if case.get("gate") else None
        if case["form"] == "train":
            s["gout"] = normal(R, H)
            s["gsum"] = normal(R, H) if case["op"] == "prenorm" else None
        return s
    S, B, H, G, K, V = (case[n] for n in "SBHGKV")
    train, step = case["form"] == "train", case["form"] == "step"
    rows = (B,) if step else (S, B)
    # q, k and v as the convolution's activation leaves them, parts of one projection's rows
    wide = torch.empty(*rows, 2 * G * K + H * V, device=DEVICE, dtype=dt)
    for part in wide.unbind(0) if not step else (wide,):
        x = torch.randn(part.shape, generator=g, device=DEVICE)
        part.copy_(x * torch.sigmoid(x))
    if not case["normalize"]:
        wide[..., :2 * G * K].mul_((0.6 * K ** 0.5) ** -1)
    s["q"] = wide[..., :G * K].unflatten(-1, (G, K))
    s["k"] = wide[..., G * K:2 * G * K].unflatten(-1, (G, K))
    s["v"] = wide[..., 2 * G * K:].unflatten(-1, (H, V))
    s["dt"], s["b"] = normal(*rows, H, scale=0.5), normal(*rows, H)
    # decay rates between 1 and 16 and step sizes between 1e-3 and 0.1, the usual start of training
    s["A"] = -uniform(H, lo=1.0, hi=16.0)
    d = torch.exp(uniform(H, lo=math.log(1e-3), hi=math.log(0.1)))
    s["dt_bias"] = torch.log(torch.expm1(d))
    s["lengths"] = None
    if case["ragged"]:
        s["lengths"] = torch.randint(0, S + 1, (B,), generator=g, device=DEVICE)
        s["lengths"][0] = S  # the longest gives the padded size
    carried = normal(B, H, K, V, scale=0.3, dtype=torch.float32)
    s["state"] = carried if not train or case["carry"] else None
    if train:
        s["gout"] = normal(*rows, H, V)
        s["gfinal"] = normal(B, H, K, V, scale=0.3, dtype=torch.float32) if case["carry"] else None
    return s


# -- the plain form ----------------------------------------------------------------------------------
def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-torch.abs(v)))


def _silu(v):
    return v * torch.sigmoid(v)


CHUNK = 64


def _chunks(v, n):
    """[S,B,H,...] as chunks [n,B,H,CHUNK,...], zeros behind the last row."""
    pad = torch.zeros((n * CHUNK - v.shape[0], *v.shape[1:]), device=v.device, dtype=v.dtype)
    return torch.cat([v, pad]).unflatten(0, (n, CHUNK)).movedim(1, 3).contiguous()


def _rows(v, S):
    """The inverse of _chunks."""
    return v.movedim(3, 1).flatten(0, 1)[:S]


def _inverse(L):
    """(I + L)^-1 for strictly lower triangular blocks [...,CHUNK,CHUNK], by halves: the lower left
    quarter of [[P, 0], [Q, R]]^-1 is -R^-1 Q P^-1."""
    eye = torch.eye(CHUNK, device=L.device)
    X = eye.expand_as(L).clone()
    at, b = torch.arange(CHUNK, device=L.device), 1
    while b < CHUNK:
        pair = at // (2 * b)
        quarter = (pair[:, None] == pair[None, :]) & (at[:, None] // b > at[None, :] // b)
        X = X - X @ (torch.where(quarter, L, 0.0) @ X)
        b *= 2
    return X


def _heads(v, H):
    """[...,G,K] -> [...,H,K]: every key head's values for each of its value heads."""
    return v.repeat_interleave(H // v.shape[-2], dim=-2)


def _normed(v, c, scale):
    """(scale v / |v|, the factor): in 32 bits."""
    v = v.float()
    r = torch.rsqrt((v * v).sum(-1, keepdim=True) + EPS) if c["normalize"] else torch.ones_like(v[..., :1])
    return v * (r * scale), r


def _plain_delta_step(s):
    c = s["case"]
    H, K, dt = c["H"], c["K"], s["v"].dtype
    q, k = (_heads(_normed(s[n], c, f)[0], H) for n, f in (("q", K ** -0.5), ("k", 1.0)))
    a = torch.exp(s["A"] * _softplus(s["dt"].float() + s["dt_bias"]))[..., None, None]
    S = s["state"] * a
    u = torch.sigmoid(s["b"].float())[..., None] * (s["v"].float() - (S * k[..., None]).sum(-2))
    S += k[..., None] * u[..., None, :]
    s["state"].copy_(S)
    return {"out": (S * q[..., None]).sum(-2).to(dt), "state": s["state"]}


def _plain_delta(s):
    """Chunks of 64 rows: within one, u solves a triangular system; the state goes from chunk to chunk."""
    c = s["case"]
    if c["form"] == "step":
        return _plain_delta_step(s)
    S, B, H, G, K, V = (c[n] for n in "SBHGKV")
    dt, n = s["v"].dtype, -(-S // CHUNK)
    live = torch.arange(S, device=DEVICE)[:, None].expand(S, B)
    live = live < (S if s["lengths"] is None else s["lengths"])
    on = live[..., None, None]
    q, rq = _normed(torch.where(on, s["q"].float(), 0.0), c, K ** -0.5)
    k, rk = _normed(torch.where(on, s["k"].float(), 0.0), c, 1.0)
    Q, Km, Vm = _chunks(_heads(q, H), n), _chunks(_heads(k, H), n), _chunks(
        torch.where(on, s["v"].float(), 0.0), n)
    raw = s["dt"].float() + s["dt_bias"]
    d = torch.where(live[..., None], _softplus(raw), 0.0)
    beta_rows = torch.where(live[..., None], torch.sigmoid(s["b"].float()), 0.0)
    beta = _chunks(beta_rows, n)[..., None]
    cum = torch.cumsum(_chunks(d.double() * s["A"], n), dim=-1)  # logarithms of decays: long sums in 64 bits
    lower = torch.ones((CHUNK, CHUNK), device=DEVICE, dtype=torch.bool).tril()
    M = torch.where(lower, torch.exp(torch.where(lower, cum[..., :, None] - cum[..., None, :], 0.0)).float(), 0.0)
    gamma = torch.exp(cum).float()[..., None]
    tail = torch.exp(cum[..., -1:] - cum).float()[..., None]  # from a row to the chunk's end
    whole = gamma[..., -1:, :]
    KT = Km.transpose(-1, -2).contiguous()
    strict = lower.tril(-1)
    L = torch.where(strict, beta * M * (Km @ KT), 0.0)
    X = _inverse(L)
    A = M * (Q @ KT)
    U0, W = X @ (beta * Vm), X @ (beta * gamma * Km)
    state = torch.zeros((B, H, K, V), device=DEVICE) if s["state"] is None else s["state"]
    before, U = [], []
    KT_tail = KT * tail.transpose(-1, -2)
    for i in range(n):
        before.append(state)
        u = U0[i] - W[i] @ state
        U.append(u)
        state = whole[i] * state + KT_tail[i] @ u
    S0, U = torch.stack(before), torch.stack(U)
    del before, U0, W
    out = torch.where(on, _rows((gamma * Q) @ S0 + A @ U, S), 0.0).to(dt)
    if c["form"] == "prompt":
        return {"out": out, "state": state}
    # backward: the state's gradient goes from chunk to chunk, the other way
    gO = _chunks(torch.where(on, s["gout"].float(), 0.0), n)
    direct = A.transpose(-1, -2).contiguous() @ gO
    XT = X.transpose(-1, -2).contiguous()
    Qg = (gamma * Q).transpose(-1, -2).contiguous()
    Kg = (gamma * Km).transpose(-1, -2).contiguous()
    K_tail = tail * Km
    gS = torch.zeros((B, H, K, V), device=DEVICE) if s["gfinal"] is None else s["gfinal"]
    after, Y = [None] * n, [None] * n
    for i in range(n - 1, -1, -1):
        after[i] = gS
        Y[i] = XT[i] @ (direct[i] + K_tail[i] @ gS)
        gS = whole[i] * gS + Qg[i] @ gO[i] - Kg[i] @ (beta[i] * Y[i])
    after, Y = torch.stack(after), torch.stack(Y)
    del direct, Qg, Kg, K_tail, XT
    gV = beta * Y
    UT = U.transpose(-1, -2).contiguous()
    gA_ = torch.where(lower, gO @ UT, 0.0)
    gL = torch.where(strict, -(Y @ UT), 0.0)
    S0T = S0.transpose(-1, -2).contiguous()
    P = Km @ S0
    gP = -gamma * gV
    gQK, gKK = gA_ * M, gL * beta * M
    from_state = gamma * (gO @ S0T)
    gQ = from_state + gQK @ Km
    through = tail * (U @ after.transpose(-1, -2).contiguous())
    gK = gP @ S0T + through + gQK.transpose(-1, -2) @ Q + gKK @ Km + gKK.transpose(-1, -2) @ Km
    E = gA_ * A + gL * L
    ends = (through * Km).sum(-1)
    gcum = E.double().sum(-1) - E.double().sum(-2) + (from_state * Q).sum(-1) + (gP * P).sum(-1) - ends
    gcum[..., -1] += ends.sum(-1) + (whole[..., 0] * (after * S0).sum(-1)).sum(-1)
    # beta: of beta (V - gamma P) and of L
    left = (Y * (Vm - gamma * P)).sum(-1) + (gL * torch.where(strict, M * (Km @ KT), 0.0)).sum(-1)
    glog = _rows(gcum.flip(-1).cumsum(-1).flip(-1), S)  # of A d, row by row, in 64 bits
    graw = torch.where(live[..., None], glog * s["A"] * torch.sigmoid(raw.double()), 0.0)
    gbeta = _rows(left, S) * beta_rows * (1 - beta_rows)

    def through_norm(gn, v, r, scale):
        gn = gn.unflatten(2, (G, H // G)).sum(3) * scale
        v = torch.where(on, v.float(), 0.0)
        if c["normalize"]:
            gn = r * (gn - v * (r * r * (v * gn).sum(-1, keepdim=True)))
        return torch.where(on, gn, 0.0).to(dt)

    got = {"out": out, "gq": through_norm(_rows(gQ, S), s["q"], rq, K ** -0.5),
           "gk": through_norm(_rows(gK, S), s["k"], rk, 1.0),
           "gv": torch.where(on, _rows(gV, S), 0.0).to(dt), "gdt": graw.to(dt),
           "gb": torch.where(live[..., None], gbeta, 0.0).to(dt),
           "gA": (glog * d).sum((0, 1)).float(), "gdt_bias": graw.sum((0, 1)).float()}
    if s["state"] is not None:
        got["state"], got["gstate"] = state, gS
    return got


def _plain_prenorm(s):
    c, dt = s["case"], s["x"].dtype
    x, w = s["x"].float(), s["weight"].float()
    r = x if s["scale"] is None else x * s["scale"].float()
    r = r if s["residual"] is None else s["residual"].float() + r
    rstd = torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS)
    got = {"out": (r * rstd * w).to(dt), "sum": r.to(dt)}
    if c["form"] == "train":
        g = s["gout"].float()
        gn, n = g * w, r * rstd
        gr = rstd * (gn - n * (gn * n).mean(-1, keepdim=True)) + s["gsum"].float()
        got["gw"] = (g * n).sum(0).to(dt)
        got["gx"] = (gr if s["scale"] is None else gr * s["scale"].float()).to(dt)
        if s["residual"] is not None:
            got["gresidual"] = gr.to(dt)
        if s["scale"] is not None:
            got["gscale"] = (gr * x).sum(0).to(dt)
    return got


def _plain_postnorm(s):
    c, dt = s["case"], s["x"].dtype
    groups = c["groups"]
    x = s["x"].float().unflatten(-1, (groups, -1))
    w = s["weight"].float()
    w = w.view(1, -1) if c["shared"] else w.view(groups, -1)
    rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    n = x * rstd
    z = None if s["z"] is None else s["z"].float().unflatten(-1, (groups, -1))
    gate = 1.0 if z is None else _silu(z)
    scale = 1.0 if s["scale"] is None else s["scale"].float().view(groups, -1)
    y = (n * w * gate * scale).flatten(1)
    out = (y if s["residual"] is None else s["residual"].float() + y).to(dt)
    if c["form"] == "forward":
        return {"out": out}
    g = s["gout"].float().unflatten(-1, (groups, -1))
    gn = g * scale * gate * w
    gx = rstd * (gn - n * (gn * n).mean(-1, keepdim=True))
    gw = (g * scale * gate * n).sum((0, 1) if c["shared"] else 0)
    got = {"out": out, "gx": gx.flatten(1).to(dt), "gw": gw.flatten().to(dt)}
    if z is not None:
        q = torch.sigmoid(z)
        got["gz"] = (g * scale * n * w * (q * (1 + z * (1 - q)))).flatten(1).to(dt)
    if s["scale"] is not None:
        got["gscale"] = (g * n * w * gate).sum(0).flatten().to(dt)
    return got


# -- the framework's calls ---------------------------------------------------------------------------
def _own_delta(s):
    mdc, c = _mdc(), s["case"]
    ins = (s["q"], s["k"], s["v"], s["dt"], s["b"], s["A"])
    if c["form"] == "step":
        out = mdc.delta_step(s["state"], *ins, dt_bias=s["dt_bias"], normalize=c["normalize"])
        return {"out": out, "state": s["state"]}
    args = {"dt_bias": s["dt_bias"], "normalize": c["normalize"], "lengths": s["lengths"], "state": s["state"]}
    if c["form"] == "prompt":
        out, state = mdc.delta_forward(*ins, **args, return_state=True)
        return {"out": out, "state": state}
    if s["state"] is None:
        out, saved = mdc.delta_forward(*ins, **args, return_saved=True)
    else:
        out, state, saved = mdc.delta_forward(*ins, **args, return_state=True, return_saved=True)
    g = mdc.delta_backward(s["gout"], *ins, saved, **args, gradFinalState=s["gfinal"])
    got = {"out": out, "gq": g.q, "gk": g.k, "gv": g.v, "gdt": g.dt, "gb": g.b, "gA": g.A,
           "gdt_bias": g.dt_bias}
    if s["state"] is not None:
        got["state"], got["gstate"] = state, g.state
    return got


def _own_prenorm(s):
    mdc = _mdc()
    args = {"residual": s["residual"], "scale": s["scale"], "eps": EPS}
    out, total = mdc.prenorm_forward(s["x"], s["weight"], **args, return_sum=True)
    got = {"out": out, "sum": total}
    if s["case"]["form"] == "train":
        g = mdc.prenorm_backward(s["gout"], s["x"], s["weight"], **args, gradSum=s["gsum"])
        got["gw"], got["gx"] = g.weight, g.x
        if s["residual"] is not None:
            got["gresidual"] = g.residual
        if s["scale"] is not None:
            got["gscale"] = g.scale
    return got


def _own_postnorm(s):
    mdc = _mdc()
    args = {"z": s["z"], "scale": s["scale"], "groups": s["case"]["groups"], "eps": EPS}
    out = mdc.postnorm_forward(s["x"], s["weight"], residual=s["residual"], **args)
    if s["case"]["form"] == "forward":
        return {"out": out}
    g = mdc.postnorm_backward(s["gout"], s["x"], s["weight"], **args)
    got = {"out": out, "gx": g.x, "gw": g.weight}
    if s["z"] is not None:
        got["gz"] = g.z
    if s["scale"] is not None:
        got["gscale"] = g.scale
    return got


def run(state):
    op = state["case"]["op"]
    if own:
        return {"delta": _own_delta, "prenorm": _own_prenorm, "postnorm": _own_postnorm}[op](state)
    return {"delta": _plain_delta, "prenorm": _plain_prenorm, "postnorm": _plain_postnorm}[op](state)


# -- what a pass cannot do without -------------------------------------------------------------------
def work(case):
    """Bytes: every input once, every output once. A training step counts its forward and its
    backward, each with the inputs that it reads. Operations: a product and a sum are two; the delta
    rule's are those of its recurrence. Ragged lengths are uniform, so half of the rows count on average."""
    form = case["form"]
    if case["op"] != "delta":
        n, H = 2 * case["R"] * case["H"], case["H"]
        res, scale = case["residual"], case["scale"]
        params = 2 * H * (2 if scale else 1)
        ops = case["R"] * H * 8
        if case["op"] == "prenorm":
            fwd = n * (2 + (2 if res else 1 if scale else 0)) + params
            bwd = n * (3 + (2 if res else 1) + (1 if res else 0)) + 2 * params
        else:
            gate = 1 if case["gate"] else 0
            fwd = n * (2 + gate + (1 if res else 0)) + params
            bwd = n * (3 + 2 * gate) + 2 * params
        return {"bytes": fwd, "flops": ops} if form == "forward" else {"bytes": fwd + bwd, "flops": 3 * ops}
    S, B, H, G, K, V = (case[n] for n in "SBHGKV")
    rows = S * B
    live = rows / 2 if case["ragged"] else rows
    ins = 2 * live * (2 * G * K + H * V + 2 * H) + 8 * H
    state = 4 * B * H * K * V
    ops = 7 * live * H * K * V
    if form == "train":
        carry = state if case["carry"] else 0
        grads = 2 * rows * (2 * G * K + H * V + 2 * H) + 8 * H
        return {"bytes": 2 * ins + 4 * rows * H * V + grads + 4 * carry, "flops": 3 * ops}
    return {"bytes": ins + 2 * rows * H * V + 2 * state, "flops": ops}


# -- the definition in 64 bits -----------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"delta": _exact_delta, "prenorm": _exact_prenorm, "postnorm": _exact_postnorm}[case["op"]](case, s)


def _exact_delta(case, s):
    """One row after the other, as the recurrence is written; the backward walks back over states that
    are computed again, 64 rows at a time."""
    S, B, H, G, K, V = (case[n] for n in "SBHGKV")
    f, step, train = torch.float64, case["form"] == "step", case["form"] == "train"
    pick = (lambda n: s[n][None]) if step else (lambda n: s[n])
    Qs, Ks, Vs, DT, Bs = (pick(n) for n in ("q", "k", "v", "dt", "b"))
    rate, bias = s["A"].to(f), s["dt_bias"].to(f)
    head = torch.arange(H, device=DEVICE) // (H // G)
    last = torch.full((B,), S, device=DEVICE) if s["lengths"] is None else s["lengths"]
    nil = torch.zeros((), dtype=f, device=DEVICE)

    def unit(v):
        return v / torch.sqrt((v ** 2).sum(-1, keepdim=True) + EPS) if case["normalize"] else v

    def row(t):
        """(live [B,1,1,1], d, a, beta, q, k, v) of row t, q and k for every value head."""
        d = torch.logaddexp(DT[t].to(f) + bias, nil)
        q = unit(Qs[t].to(f)).index_select(1, head) / math.sqrt(K)
        k = unit(Ks[t].to(f)).index_select(1, head)
        return ((t < last)[:, None, None, None], d, torch.exp(rate * d), 1 / (1 + torch.exp(-Bs[t].to(f))),
                q, k, Vs[t].to(f))

    def advance(state, t):
        on, d, a, beta, q, k, v = row(t)
        kept = state * a[..., None, None]
        u = beta[..., None] * (v - torch.matmul(k[..., None, :], kept)[..., 0, :])
        return torch.where(on, kept + k[..., :, None] * u[..., None, :], state)

    state = torch.zeros((B, H, K, V), dtype=f, device=DEVICE) if s["state"] is None else s["state"].to(f)
    out = torch.zeros((S, B, H, V), dtype=f, device=DEVICE)
    marks = []
    for t in range(S):
        if train and t % 64 == 0:
            marks.append(state)
        state = advance(state, t)
        on, _, _, _, q, _, _ = row(t)
        out[t] = torch.where(on[..., 0], torch.matmul(q[..., None, :], state)[..., 0, :], 0.0)
    if not train:
        return {"out": out[0] if step else out, "state": state}
    got = {"out": out, "gq": torch.zeros(Qs.shape, dtype=f, device=DEVICE), "gk": torch.zeros(Ks.shape, dtype=f, device=DEVICE),
           "gv": torch.zeros(Vs.shape, dtype=f, device=DEVICE), "gdt": torch.zeros(DT.shape, dtype=f, device=DEVICE),
           "gb": torch.zeros(Bs.shape, dtype=f, device=DEVICE), "gA": torch.zeros(H, dtype=f, device=DEVICE),
           "gdt_bias": torch.zeros(H, dtype=f, device=DEVICE)}
    gs = torch.zeros_like(state) if s["gfinal"] is None else s["gfinal"].to(f)
    if s["state"] is not None:
        got["state"] = state

    def unit_back(gn, v, factor):
        """The gradient of the raw rows: gn is that of factor * unit(v), for every value head."""
        gn = factor * gn.view(B, G, H // G, K).sum(2)
        if not case["normalize"]:
            return gn
        v = v.to(f)
        size = torch.sqrt((v ** 2).sum(-1, keepdim=True) + EPS)
        return gn / size - v * ((gn * v).sum(-1, keepdim=True) / size ** 3)

    for block in range(len(marks) - 1, -1, -1):
        lo, hi = 64 * block, min(S, 64 * block + 64)
        states = [marks.pop()]
        for t in range(lo, hi):
            states.append(advance(states[-1], t))
        for t in range(hi - 1, lo - 1, -1):
            on, d, a, beta, q, k, v = row(t)
            on1, on2 = on[..., 0, 0], on[..., 0]
            new, old = states[t - lo + 1], states[t - lo]
            go = torch.where(on2, s["gout"][t].to(f), 0.0)
            g = gs + q[..., :, None] * go[..., None, :]
            kept = old * a[..., None, None]
            rest = v - torch.matmul(k[..., None, :], kept)[..., 0, :]
            gu = torch.matmul(k[..., None, :], g)[..., 0, :]
            gq = torch.matmul(new, go[..., :, None])[..., 0]
            gk = torch.matmul(g, (beta[..., None] * rest)[..., :, None])[..., 0]
            gv = beta[..., None] * gu
            gk = gk - torch.matmul(kept, gv[..., :, None])[..., 0]
            gkept = g - k[..., :, None] * gv[..., None, :]
            glog = torch.where(on1, (gkept * kept).sum((-1, -2)), 0.0)
            gbeta = (gu * rest).sum(-1)
            got["gq"][t] = torch.where(on2, unit_back(gq, Qs[t], 1 / math.sqrt(K)), 0.0)
            got["gk"][t] = torch.where(on2, unit_back(gk, Ks[t], 1.0), 0.0)
            got["gv"][t] = torch.where(on2, gv, 0.0)
            got["gb"][t] = torch.where(on1, gbeta * beta * (1 - beta), 0.0)
            raw = glog * rate / (1 + torch.exp(-(DT[t].to(f) + bias)))
            got["gdt"][t] = raw
            got["gdt_bias"] += raw.sum(0)
            got["gA"] += (glog * d).sum(0)
            gs = torch.where(on, gkept * a[..., None, None], gs)
    if s["state"] is not None:
        got["gstate"] = gs
    return got


def _exact_prenorm(case, s):
    f, H = torch.float64, case["H"]
    one, nil = torch.ones(H, dtype=f, device=DEVICE), torch.zeros((), dtype=f, device=DEVICE)
    x, w = s["x"].to(f), s["weight"].to(f)
    scale = one if s["scale"] is None else s["scale"].to(f)
    r = torch.addcmul(nil if s["residual"] is None else s["residual"].to(f), x, scale)
    size = torch.sqrt(torch.linalg.vector_norm(r, dim=1, keepdim=True) ** 2 / H + EPS)
    got = {"out": w * r / size, "sum": r}
    if case["form"] == "train":
        g = s["gout"].to(f)
        along = torch.mv(g * r, w)[:, None]
        gr = s["gsum"].to(f) + (g * w) / size - r * along / (H * size ** 3)
        got["gw"], got["gx"] = (g * r / size).sum(0), gr * scale
        if s["residual"] is not None:
            got["gresidual"] = gr
        if s["scale"] is not None:
            got["gscale"] = (gr * x).sum(0)
    return got


def _exact_postnorm(case, s):
    """Group by group."""
    f, H, groups = torch.float64, case["H"], case["groups"]
    D = H // groups
    parts = {n: [] for n in ("out", "gx", "gw", "gz", "gscale")}
    for i in range(groups):
        at = slice(i * D, (i + 1) * D)
        x = s["x"][:, at].to(f)
        w = (s["weight"] if case["shared"] else s["weight"][at]).to(f)
        scale = torch.ones(D, dtype=f, device=DEVICE) if s["scale"] is None else s["scale"][at].to(f)
        size = torch.sqrt(torch.linalg.vector_norm(x, dim=1, keepdim=True) ** 2 / D + EPS)
        gate, slope = torch.ones_like(x), None
        if s["z"] is not None:
            z = s["z"][:, at].to(f)
            e = torch.exp(-z)
            gate, slope = z / (1 + e), (1 + e + z * e) / (1 + e) ** 2
        y = scale * (w * x / size * gate)
        parts["out"].append(y if s["residual"] is None else s["residual"][:, at].to(f) + y)
        if case["form"] == "forward":
            continue
        g = s["gout"][:, at].to(f)
        inner = g * gate * scale * w
        parts["gx"].append(inner / size - x * (inner * x).sum(1, keepdim=True) / (D * size ** 3))
        parts["gw"].append((g * gate * scale * x / size).sum(0))
        if slope is not None:
            parts["gz"].append(g * scale * w * slope * x / size)
        if s["scale"] is not None:
            parts["gscale"].append((g * gate * w * x / size).sum(0))
    got = {n: torch.cat(v, -1) for n, v in parts.items() if v}
    if case["form"] == "train" and case["shared"]:
        got["gw"] = sum(parts["gw"])
    return got
