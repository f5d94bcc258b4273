"""Plain 64-bit forms of the state space block's operators on the CPU, row by row as the formulas are
written, for the tests. Each function also gives, for every result, the same sum with every term
taken absolutely ("mag"): what an error bound is relative to."""
from __future__ import annotations

import numpy as np
import torch

F = torch.float64


def sigmoid(v):
    return torch.where(v >= 0, 1 / (1 + torch.exp(-v.clamp(min=0))),
                       torch.exp(v.clamp(max=0)) / (1 + torch.exp(v.clamp(max=0))))


def softplus(v):
    return v.clamp(min=0) + torch.log1p(torch.exp(-v.abs()))


def act(v, kind):
    if kind == "relu":
        return v.clamp(min=0)
    if kind == "silu":
        return v * sigmoid(v)
    if kind == "gelu":
        return 0.5 * v * (1 + torch.tanh((2 / np.pi) ** 0.5 * (v + 0.044715 * v ** 3)))
    return softplus(v) if kind == "softplus" else v


def act_slope(v, kind):
    if kind == "relu":
        return (v > 0).to(v.dtype)
    if kind == "silu":
        g = sigmoid(v)
        return g + v * g * (1 - g)
    if kind == "gelu":
        c = (2 / np.pi) ** 0.5
        t = torch.tanh(c * (v + 0.044715 * v ** 3))
        return 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * c * (1 + 3 * 0.044715 * v * v)
    return sigmoid(v) if kind == "softplus" else torch.ones_like(v)


def lens_of(lengths, S, B):
    return [S] * B if lengths is None else [min(max(int(n), 0), S) for n in lengths]


def conv(x, w, bias, kind, lengths=None, state=None, gy=None, gfinal=None):
    """dict of y, final state and (with gy) gradients, each as (value, mag). Dead rows of the inputs
    are never read."""
    x, w = x.to(F), w.to(F)
    S, B, H = x.shape
    W = w.shape[0]
    bias = torch.zeros(H, dtype=F) if bias is None else bias.to(F)
    state = torch.zeros((W - 1, B, H), dtype=F) if state is None else state.to(F)
    y, ymag = torch.zeros((S, B, H), dtype=F), torch.zeros((S, B, H), dtype=F)
    final = torch.zeros((W - 1, B, H), dtype=F)
    g = {k: torch.zeros(s, dtype=F) for k, s in
         (("gx", (S, B, H)), ("gw", (W, H)), ("gb", (H,)), ("gs", (W - 1, B, H)))}
    gm = {k: torch.zeros_like(v) for k, v in g.items()}
    for b, n in enumerate(lens_of(lengths, S, B)):
        rows = torch.cat([state[:, b], x[:n, b]])  # row t of x at t + W - 1
        final[:, b] = rows[n:]
        gr, grm = torch.zeros_like(rows), torch.zeros_like(rows)
        if gfinal is not None:
            gr[n:] += gfinal[:, b].to(F)
            grm[n:] += gfinal[:, b].to(F).abs()
        for t in range(n):
            pre = bias + (w * rows[t:t + W]).sum(0)
            premag = bias.abs() + (w * rows[t:t + W]).abs().sum(0)
            y[t, b] = act(pre, kind)
            ymag[t, b] = premag
            if gy is not None:
                go = gy[t, b].to(F)
                q = go * act_slope(pre, kind)
                qm = go.abs() * (1.1 + premag)  # slopes are below 1.1, their slope below 1
                gr[t:t + W] += q * w
                grm[t:t + W] += qm * w.abs()
                g["gw"] += q * rows[t:t + W]
                gm["gw"] += qm * rows[t:t + W].abs()
                g["gb"] += q
                gm["gb"] += qm
        g["gs"][:, b], gm["gs"][:, b] = gr[:W - 1], grm[:W - 1]
        g["gx"][:n, b], gm["gx"][:n, b] = gr[W - 1:], grm[W - 1:]
    out = {"y": (y, ymag), "state": (final, final.abs())}
    if gy is not None:
        out |= {k: (g[k], gm[k]) for k in g}
    return out


def scan(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, use_softplus=True, lengths=None, state=None,
         gout=None, gfinal=None):
    """As conv: out, final state and gradients with their magnitudes."""
    S, B, H = x.shape
    N, G = A.shape[0], Bm.shape[2]
    A = A.to(F)
    D = torch.zeros(H, dtype=F) if D is None else D.to(F)
    bias = torch.zeros(H, dtype=F) if dt_bias is None else dt_bias.to(F)
    grp = torch.arange(H) // (H // G)
    zero = lambda *s: torch.zeros(s, dtype=F)  # noqa: E731
    out, outm = zero(S, B, H), zero(S, B, H)
    final, finalm = zero(B, N, H), zero(B, N, H)
    names = {"gx": (S, B, H), "gdt": (S, B, H), "gz": (S, B, H), "gB": (S, B, G, N),
             "gC": (S, B, G, N), "gA": (N, H), "gD": (H,), "gbias": (H,), "gs": (B, N, H)}
    g = {k: zero(*s) for k, s in names.items()}
    gm = {k: zero(*s) for k, s in names.items()}
    to_groups = lambda v: v.reshape(N, G, H // G).sum(2).t()  # noqa: E731
    for b, n in enumerate(lens_of(lengths, S, B)):
        s = zero(N, H) if state is None else state[b].to(F)
        sm = s.abs()
        kept = [(s, sm)]
        for t in range(n):
            v = dt[t, b].to(F) + bias
            d = softplus(v) if use_softplus else v
            xt, Bt, Ct = x[t, b].to(F), Bm[t, b].to(F)[grp].t(), Cm[t, b].to(F)[grp].t()
            a = torch.exp(d * A)
            s = a * s + d * xt * Bt
            sm = a * sm + (d * xt * Bt).abs()
            kept.append((s, sm))
            y, ym = (Ct * s).sum(0) + D * xt, (Ct.abs() * sm).sum(0) + (D * xt).abs()
            if z is not None:
                gate = act(z[t, b].to(F), "silu")
                y, ym = y * gate, ym * gate.abs()
            out[t, b], outm[t, b] = y, ym
        final[b], finalm[b] = s, sm
        if gout is None:
            continue
        c = zero(N, H) if gfinal is None else gfinal[b].to(F)
        cm = c.abs()
        for t in range(n - 1, -1, -1):
            v = dt[t, b].to(F) + bias
            d, slope = (softplus(v), sigmoid(v)) if use_softplus else (v, torch.ones_like(v))
            xt, Bt, Ct = x[t, b].to(F), Bm[t, b].to(F)[grp].t(), Cm[t, b].to(F)[grp].t()
            a, go = torch.exp(d * A), gout[t, b].to(F)
            (s, sm), (s0, s0m) = kept[t + 1], kept[t]
            gy = go
            if z is not None:
                zt = z[t, b].to(F)
                y, ym = (Ct * s).sum(0) + D * xt, (Ct.abs() * sm).sum(0) + (D * xt).abs()
                g["gz"][t, b] = go * y * act_slope(zt, "silu")
                gm["gz"][t, b] = go.abs() * ym * (1.1 + zt.abs())
                gy = go * act(zt, "silu")
            gs, gsm = c + Ct * gy, cm + (Ct * gy).abs()
            g["gC"][t, b], gm["gC"][t, b] = to_groups(gy * s), to_groups(gy.abs() * sm)
            g["gB"][t, b] = to_groups(gs * d * xt)
            gm["gB"][t, b] = to_groups(gsm * (d * xt).abs())
            u, um = (gs * Bt).sum(0), (gsm * Bt.abs()).sum(0)
            c, cm = gs * a, gsm * a
            q, qm = c * s0, cm * s0m
            g["gx"][t, b], gm["gx"][t, b] = u * d + D * gy, um * d.abs() + (D * gy).abs()
            gd = ((q * A).sum(0) + u * xt) * slope
            gdm = ((qm * A.abs()).sum(0) + um * xt.abs()) * (slope + v.abs())
            g["gdt"][t, b], gm["gdt"][t, b] = gd, gdm
            for k, val, mag in (("gA", q * d, qm * d.abs()), ("gD", gy * xt, (gy * xt).abs()),
                                ("gbias", gd, gdm)):
                g[k] += val
                gm[k] += mag
        g["gs"][b], gm["gs"][b] = c, cm
    res = {"out": (out, outm), "state": (final, finalm)}
    if gout is not None:
        res |= {k: (g[k], gm[k]) for k in g}
    return res


def close(got, ref, slack, name):
    """|got - value| <= half a step of got's type at the value + slack * mag (+ half the subnormal
    step where the value is that small)."""
    value, mag = ref
    fi = torch.finfo(got.dtype)
    half = fi.eps / 2 if got.dtype != torch.float32 else 0.0
    tiny = fi.tiny * fi.eps / 2
    got = got.detach().cpu().to(F)
    assert got.shape == value.shape, (name, got.shape, value.shape)
    assert torch.isfinite(got).all(), f"{name}: not finite"
    tol = half * value.abs() + slack * mag * (1 + half) + tiny
    off = (got - value).abs() - tol
    if off.numel() and float(off.max()) > 0:
        at = int(off.argmax())
        raise AssertionError(f"{name}: {int((off > 0).sum())} of {off.numel()} off, worst at flat {at}: "
                             f"{got.flatten()[at]} for {value.flatten()[at]} +- {tol.flatten()[at]}")
