"""The selective scan in 64 bits with, beside every value, a bound of what fp32 arithmetic in the kernels'
order may be off by, carried through the recurrences (first-order terms; 5 % for the others).

Units: u = 2^-24, half a step of fp32. exp2 and the reciprocal are the hardware's, within one step; FN =
2^-22 for each leaves another. Of a step size d = softplus(v), v = dt + dt_bias:

    v        u |v|                                    one addition
    d        slope u |v| + d (2 u max(-v, 0) + 2^-21)  exp of -|v| log2 e, whose product and constant are
                                                      rounded, and log(1+e) to 2^-22 of itself
    sigmoid  2 u |v| + 2^-20, relative                exp, 1 + e, reciprocal
    a        a (|A| err(d) + 3 u |d A| + FN)          exp2 of d times A log2 e

A state adds a's error times the last state, d x B's and one rounding; sums over up to 32 states are four
in a lane and up to eight waves', with D x 14 roundings; sums over channels six joins of 64 lanes (then
fp64); gA 16 rows (then fp64); gD and gdt_bias each 16th row of 512, then those sums. Where the rows are
cut into chunks, the state at a chunk's start is exp(A sum d) times the one before, whose sum of n terms
is off by n u of itself: n u x exp(-x) <= 0.4 n u of that state, over all chunks 0.4 S u of the largest."""
from __future__ import annotations

import torch

from . import ssm_ref as ref

F = torch.float64
U, FN = 2.0 ** -24, 2.0 ** -22


def softplus(v):
    d, slope = ref.softplus(v), ref.sigmoid(v)
    return d, slope * U * v.abs() + d * (2 * U * (-v).clamp(min=0) + 2.0 ** -21), slope


def sigmoid_err(v, g):
    return g * (2 * U * v.abs() + 2.0 ** -20)


def scan(x, dt, A, Bm, Cm, D, z, dt_bias, lengths, state, gout, gfinal, chunked=False, held=None):
    """{name: (value, bound)} of the forward's and backward's results. `held`: a type that the state is
    rounded to after every row, to see whether the bounds notice."""
    S, B, H = x.shape
    N, G = A.shape[0], Bm.shape[2]
    A = A.to(F)
    D = torch.zeros(H, dtype=F) if D is None else D.to(F)
    bias = torch.zeros(H, dtype=F) if dt_bias is None else dt_bias.to(F)
    grp = torch.arange(H) // (H // G)
    zero = lambda *s: torch.zeros(s, dtype=F)  # noqa: E731
    shapes = {"out": (S, B, H), "state": (B, N, H), "gx": (S, B, H), "gdt": (S, B, H), "gz": (S, B, H),
              "gB": (S, B, G, N), "gC": (S, B, G, N), "gA": (N, H), "gD": (H,), "gbias": (H,),
              "gs": (B, N, H)}
    val, err = ({k: zero(*s) for k, s in shapes.items()} for _ in range(2))
    groups = lambda v: v.reshape(N, G, H // G).sum(2).t()  # noqa: E731
    fold = 0.4 * S * U if chunked else 0.0
    few = (36 + S / 512) * U
    for b, n in enumerate(ref.lens_of(lengths, S, B)):
        s = zero(N, H) if state is None else state[b].to(F)
        es, most = torch.zeros_like(s), s.abs()
        rows = []
        for t in range(n):
            v = dt[t, b].to(F) + bias
            d, ed, slope = softplus(v)
            xt, Bt, Ct = x[t, b].to(F), Bm[t, b].to(F)[grp].t(), Cm[t, b].to(F)[grp].t()
            a, dx = torch.exp(d * A), d * xt
            ea = a * (A.abs() * ed + 3 * U * (d * A).abs() + FN)
            edx = xt.abs() * ed + U * dx.abs()
            before = (s, es + fold * most)
            es = a * es + ea * s.abs() + edx * Bt.abs() + 2 * U * (dx * Bt).abs()
            s = a * s + dx * Bt
            if held is not None:
                s = s.to(held).to(F)
            es = es + U * s.abs()
            most = torch.maximum(most, s.abs())
            e = es + fold * most
            y = (Ct * s).sum(0) + D * xt
            ey = (Ct.abs() * e).sum(0) + 14 * U * ((Ct * s).abs().sum(0) + (D * xt).abs())
            gate, egate = torch.ones(H, dtype=F), zero(H)
            if z is not None:
                zt = z[t, b].to(F)
                g = ref.sigmoid(zt)
                gate, egate = zt * g, zt.abs() * (sigmoid_err(zt, g) + U * g)
            val["out"][t, b] = y * gate
            err["out"][t, b] = ey * gate.abs() + y.abs() * egate + U * (y * gate).abs()
            rows.append((d, ed, slope, v, xt, Bt, Ct, a, ea, dx, edx, before, (s, e), y, ey, gate, egate))
        val["state"][b], err["state"][b] = s, es + fold * most
        c = zero(N, H) if gfinal is None else gfinal[b].to(F)
        ec, most = torch.zeros_like(c), c.abs()
        for t in range(n - 1, -1, -1):
            (d, ed, slope, v, xt, Bt, Ct, a, ea, dx, edx, (s0, es0), (s, e), y, ey, gate, egate) = rows[t]
            go = gout[t, b].to(F)
            gy, egy = go * gate, go.abs() * egate + (U * (go * gate).abs() if z is not None else 0.0)
            if z is not None:
                zt = z[t, b].to(F)
                g = ref.sigmoid(zt)
                ss = ref.act_slope(zt, "silu")
                ess = 2 * sigmoid_err(zt, g) * (1 + zt.abs()) + 2 * U * (1 + zt.abs()) * g
                val["gz"][t, b] = go * y * ss
                err["gz"][t, b] = go.abs() * (ss.abs() * ey + y.abs() * ess) + 3 * U * (go * y * ss).abs()
            gs = Ct * gy + c
            egs = Ct.abs() * egy + ec + fold * most + U * gs.abs()
            val["gC"][t, b] = groups(gy * s)
            err["gC"][t, b] = groups(gy.abs() * e + egy * s.abs() + 8 * U * (gy * s).abs())
            val["gB"][t, b] = groups(gs * dx)
            err["gB"][t, b] = groups(gs.abs() * edx + egs * dx.abs() + 8 * U * (gs * dx).abs())
            u = (gs * Bt).sum(0)
            eu = (egs * Bt.abs() + 14 * U * (gs * Bt).abs()).sum(0)
            ec = a * (Ct.abs() * egy + ec + U * gs.abs()) + gs.abs() * ea
            c = gs * a
            ec = ec + U * c.abs()
            most = torch.maximum(most, c.abs())
            q = c * s0
            eq = c.abs() * es0 + s0.abs() * (ec + fold * most) + U * q.abs()
            w = (q * A).sum(0)
            ew = (eq * A.abs() + 18 * U * (q * A).abs()).sum(0)
            gd = w + u * xt
            egd = ew + xt.abs() * eu + 2 * U * (w.abs() + (u * xt).abs())
            gdt = gd * slope
            egdt = slope * egd + gd.abs() * slope * (3 * U * v.abs() + 2.0 ** -20) + U * gdt.abs()
            val["gdt"][t, b], err["gdt"][t, b] = gdt, egdt
            val["gx"][t, b] = u * d + D * gy
            err["gx"][t, b] = (d * eu + u.abs() * ed + D.abs() * egy +
                               2 * U * ((u * d).abs() + (D * gy).abs()))
            val["gA"] += q * d
            err["gA"] += eq * d + q.abs() * ed + 18 * U * (q * d).abs()
            val["gD"] += gy * xt
            err["gD"] += egy * xt.abs() + few * (gy * xt).abs()
            val["gbias"] += gdt
            err["gbias"] += egdt + few * gdt.abs()
        val["gs"][b], err["gs"][b] = c, ec + fold * most
    for k in ("gA", "gD", "gbias", "state", "gs"):
        err[k] += U * val[k].abs()
    return {k: (val[k], 1.05 * err[k] + 2.0 ** -120) for k in val}
