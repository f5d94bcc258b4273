"""Plain 64-bit forms of the gated delta rule and of the norms around a block on the CPU, as the formulas are
written, for the tests."""
from __future__ import annotations

import torch

from .ssm_ref import F, lens_of, sigmoid, softplus

EPS = 1e-6


def unit(v, normalize):
    return v / torch.sqrt((v * v).sum(-1, keepdim=True) + EPS) if normalize else v


def unit_back(g, v, normalize):
    if not normalize:
        return g
    size = torch.sqrt((v * v).sum(-1, keepdim=True) + EPS)
    return g / size - v * (g * v).sum(-1, keepdim=True) / size ** 3


def before_back(g, v, normalize):
    """The size of what unit_back subtracts from."""
    return g / torch.sqrt((v * v).sum(-1, keepdim=True) + EPS) if normalize else g


def delta(q, k, v, dt, b, A, dt_bias=None, use_softplus=True, normalize=True, scale=None, lengths=None,
          state=None, gout=None, gfinal=None):
    """dict of out, state and (with gout) gradients; gq_before and gk_before are those of q and k without what they
    lose along the row itself, glog is the largest gradient of a row's log decay, a head
    each, and steps the sum of its step sizes. Rows past a length are never read."""
    S, B, G, K = q.shape
    H, V = v.shape[-2:]
    head = torch.arange(H) // (H // G)
    scale = K ** -0.5 if scale is None else scale
    A = A.to(F)
    bias = torch.zeros(H, dtype=F) if dt_bias is None else dt_bias.to(F)
    z = lambda *s: torch.zeros(s, dtype=F)  # noqa: E731
    r = {"out": z(S, B, H, V), "state": z(B, H, K, V)}
    if gout is not None:
        r |= {"gq": z(S, B, G, K), "gk": z(S, B, G, K), "gv": z(S, B, H, V), "gdt": z(S, B, H), "gb": z(S, B, H),
              "gA": z(H), "gdt_bias": z(H), "gstate": z(B, H, K, V), "glog": z(H), "steps": z(H), "gq_before": z(S, B, G, K),
              "gk_before": z(S, B, G, K)}
    for i, n in enumerate(lens_of(lengths, S, B)):
        s = z(H, K, V) if state is None else state[i].to(F).clone()
        kept, rows = [], []
        for t in range(n):
            raw = dt[t, i].to(F) + bias
            d, slope = (softplus(raw), sigmoid(raw)) if use_softplus else (raw, torch.ones_like(raw))
            a = torch.where(d == 0, 1.0, torch.exp(A * d))
            beta = sigmoid(b[t, i].to(F))
            qn, kn = unit(q[t, i].to(F), normalize)[head] * scale, unit(k[t, i].to(F), normalize)[head]
            kept.append(s)
            s = s * a[:, None, None]
            rest = v[t, i].to(F) - torch.einsum("hk,hkv->hv", kn, s)
            u = beta[:, None] * rest
            s = s + kn[:, :, None] * u[:, None, :]
            r["out"][t, i] = torch.einsum("hk,hkv->hv", qn, s)
            rows.append((d, slope, a, beta, qn, kn, rest, u, s))
        r["state"][i] = s
        if gout is None:
            continue
        gs = z(H, K, V) if gfinal is None else gfinal[i].to(F).clone()
        for t in range(n - 1, -1, -1):
            d, slope, a, beta, qn, kn, rest, u, s = rows[t]
            go = gout[t, i].to(F)
            gq = torch.einsum("hkv,hv->hk", s, go) * scale
            gs = gs + qn[:, :, None] * go[:, None, :]
            gu = torch.einsum("hk,hkv->hv", kn, gs)
            gv = beta[:, None] * gu
            faded = kept[t] * a[:, None, None]
            gk = torch.einsum("hkv,hv->hk", gs, u) - torch.einsum("hkv,hv->hk", faded, gv)
            gs = gs - kn[:, :, None] * gv[:, None, :]
            glog = (gs * faded).sum((1, 2))
            gs = gs * a[:, None, None]
            r["gv"][t, i] = gv
            r["gb"][t, i] = (gu * rest).sum(-1) * beta * (1 - beta)
            r["gdt"][t, i] = glog * A * slope
            r["gA"] += glog * d
            r["gdt_bias"] += glog * A * slope
            r["glog"] = torch.maximum(r["glog"], glog.abs())
            r["steps"] += d.abs()
            groups = lambda g: z(G, K).index_add_(0, head, g)  # noqa: E731
            for name, grad, row in (("gq", groups(gq), q[t, i].to(F)), ("gk", groups(gk), k[t, i].to(F))):
                r[name][t, i] = unit_back(grad, row, normalize)
                r[name + "_before"][t, i] = before_back(grad, row, normalize)
        r["gstate"][i] = gs
    return r


def prenorm(x, weight, residual=None, scale=None, eps=EPS, gout=None, gsum=None):
    """dict of (value, mag), mag with every term taken absolutely."""
    x, w = x.to(F), weight.to(F)
    H = x.shape[-1]
    res = torch.zeros_like(x) if residual is None else residual.to(F)
    sc = torch.ones(H, dtype=F) if scale is None else scale.to(F)
    s, sm = res + sc * x, res.abs() + (sc * x).abs()
    size = torch.sqrt((s * s).mean(-1, keepdim=True) + eps)
    r = {"out": (s / size * w, sm / size * w.abs()), "sum": (s, sm)}
    if gout is not None:
        g = gout.to(F)
        gn, n, nm = g * w, s / size, sm / size
        mean, meanm = (gn * n).mean(-1, keepdim=True), (gn * nm).abs().mean(-1, keepdim=True)
        gr, grm = (gn - n * mean) / size, (gn.abs() + nm * meanm) / size
        if gsum is not None:
            gr, grm = gr + gsum.to(F), grm + gsum.to(F).abs()
        over = tuple(range(x.dim() - 1))
        r |= {"gx": (gr * sc, grm * sc.abs()), "gresidual": (gr, grm), "gw": ((g * n).sum(over), (g * nm).abs().sum(over)),
              "gscale": ((gr * x).sum(over), (grm * x.abs()).sum(over))}
    return r


def postnorm(x, weight, z=None, residual=None, scale=None, groups=1, eps=EPS, gout=None):
    x = x.to(F)
    H = x.shape[-1]
    shared = weight.shape[0] != H
    w = weight.to(F).repeat(groups) if shared else weight.to(F)
    sc = torch.ones(H, dtype=F) if scale is None else scale.to(F)
    part = lambda t: t.unflatten(-1, (groups, H // groups))  # noqa: E731
    size = torch.sqrt((part(x) ** 2).mean(-1, keepdim=True) + eps).expand(part(x).shape).flatten(-2)
    n = x / size
    zz = None if z is None else z.to(F)
    gate = torch.ones_like(x) if z is None else zz * sigmoid(zz)
    y = n * w * gate * sc
    res = torch.zeros_like(x) if residual is None else residual.to(F)
    r = {"out": (res + y, res.abs() + y.abs())}
    if gout is not None:
        g = gout.to(F)
        gn = g * w * gate * sc
        mean = part(gn * n).mean(-1, keepdim=True).expand(part(x).shape).flatten(-2)
        meanm = part(gn * n).abs().mean(-1, keepdim=True).expand(part(x).shape).flatten(-2)
        over = tuple(range(x.dim() - 1))
        gw, gwm = (g * n * gate * sc).sum(over), (g * n * gate * sc).abs().sum(over)
        if shared:
            gw, gwm = part(gw).sum(0), part(gwm).sum(0)
        r |= {"gx": ((gn - n * mean) / size, (gn.abs() + (n * meanm).abs()) / size), "gw": (gw, gwm),
              "gscale": ((g * n * w * gate).sum(over), (g * n * w * gate).abs().sum(over))}
        if z is not None:
            q = sigmoid(zz)
            slope = q + zz * q * (1 - q)
            r["gz"] = (g * n * w * sc * slope, (g * n * w * sc).abs() * (1.1 + zz.abs()))
    return r


def norm_close(got, value, tol, name, mag=None):
    """The 2-norm of the difference against that of the value (or `mag`), and every difference against 16 times as
    much of the root mean square or the value itself. `tol` excludes the result's rounding."""
    fi = torch.finfo(got.dtype)
    half = fi.eps / 2 if got.dtype != torch.float32 else 0.0
    got = got.detach().cpu().to(F)
    assert got.shape == value.shape, (name, got.shape, value.shape)
    assert torch.isfinite(got).all(), f"{name}: not finite"
    if not value.numel():
        return
    size = value.norm() if mag is None else torch.as_tensor(mag, dtype=F)
    off = (got - value).norm()
    tiny = fi.tiny * value.numel() ** 0.5
    assert off <= half * value.norm() + tol * size + tiny, f"{name}: {float(off)} of {float(size)}: {float(off / size)}"
    rms = size / value.numel() ** 0.5
    far = (got - value).abs() - half * value.abs() - 16 * tol * (rms + value.abs()) - fi.tiny
    assert float(far.max()) <= 0, f"{name}: worst at flat {int(far.argmax())}, {float(got.flatten()[far.argmax()])} for " \
                                  f"{float(value.flatten()[far.argmax()])}"
