"""Gated delta rule against the 64-bit form.

Tolerances, in the 2-norm, for sequences of c = ceil(S / 64) chunks. A chunk's result passes some eight products and
scalings on its way to the next one, each with a relative error of at most 2^-21 (two terms of 11 bits each: 2^-22 of
either operand, and fp32 sums), which is 2^-18 a chunk; the step itself does not grow a state (decays and I - beta k k^T
are contractions for normalized keys), so errors add: (c + 4) 2^-18 for states and gradients, besides a 16-bit
result's own rounding of half a step. bf16 outputs are made of one fp16 term of S0, A and U (2^-12 each on the average
of a value), whose parts are up to four times the result: 3 * 4 * 2^-12. Gradients of A and dt_bias add a row's step size
times the gradient of its log decay: they are compared with the sum of the steps times the largest of those. The gradient
of a row of q or k is g / |k| less its part along the row: two terms that are right to the bound, and whose difference may
be far smaller than either (all of it, for K = 1), so that the bound is relative to g / |k|. What a chunk hands on of the
state that it got (or backwards of the state's gradient) may have faded below what the two terms keep of a column: they
lose up to 2^-40 of the largest value in it, in each of 64 rows, whose factors are at most 1: 2^-34 of what came in."""
from __future__ import annotations

import pytest
import torch

import masked_depthwise_causal_amd as mdc

from . import delta_ref as ref
from .gpu_util import announce
from .ssm_ref import lens_of
from .test_conv_act import DT, dirty

pytestmark = pytest.mark.gpu


def slack(S):
    return ((S + 63) // 64 + 4) * 2.0 ** -18


def faded(value, came, e):
    """The size that the bound e is relative to, for what is left of `came`."""
    return value.norm() + (0 if came is None else came.double().norm() * 2.0 ** -34 / e)


def inputs(S, B, H, G, K, V, dtype, seed, bias=True, state=True, unit=True):
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    size = 1.0 if unit else K ** -0.5
    v = {"q": (r(S, B, G, K) * size).to(dt), "k": (r(S, B, G, K) * size).to(dt), "v": r(S, B, H, V).to(dt),
         "dt": (r(S, B, H) * 0.5).to(dt), "b": r(S, B, H).to(dt), "A": -torch.rand(H, generator=g) * 8 - 0.2,
         "dt_bias": r(H) - 2.5 if bias else None, "state": r(B, H, K, V) if state else None}
    return v, r(S, B, H, V).to(dt), r(B, H, K, V) if state else None


def place(v, layout):
    """The device copies of q, k, v in a layout: contiguous, parts of one wider row, or batch first."""
    q, k, x = (v[n] for n in ("q", "k", "v"))
    if layout == "contig":
        return q.cuda(), k.cuda(), x.cuda()
    if layout == "parts":
        wide = torch.cat([t.flatten(2) for t in (q, k, x)] + [torch.zeros(*q.shape[:2], 5, dtype=q.dtype)], -1).cuda()
        at, out = 0, []
        for t in (q, k, x):
            n = t.shape[2] * t.shape[3]
            out.append(wide[..., at:at + n].unflatten(-1, t.shape[2:]))
            at += n
        return tuple(out)
    return tuple(t.transpose(0, 1).contiguous().cuda().transpose(0, 1) for t in (q, k, x))


def check(S, B, H, G, K, V, dtype, lengths=None, layout="contig", normalize=True, softplus=True, scale=None, seed=0,
          change=None, **parts):
    v, go, gf = inputs(S, B, H, G, K, V, dtype, seed, unit=normalize, **parts)
    if not softplus:  # dt and its bias are then the step size itself
        v["dt"], v["dt_bias"] = v["dt"].abs() * 0.2, None if v["dt_bias"] is None else v["dt_bias"].abs() * 0.1
    if change:
        change(v, go)
    r = ref.delta(v["q"], v["k"], v["v"], v["dt"], v["b"], v["A"], v["dt_bias"], softplus, normalize, scale, lengths,
                  v["state"], go, gf)
    for b, n in enumerate(lens_of(lengths, S, B)):  # what dead rows hold must not matter
        for name in ("q", "k", "v", "dt", "b"):
            v[name][n:, b] = float("nan")
        go[n:, b] = float("inf")
    q, k, x = place(v, layout)
    dev = {n: None if v[n] is None else v[n].cuda() for n in ("dt", "b", "A", "dt_bias", "state")}
    ins = (q, k, x, dev["dt"], dev["b"], dev["A"])
    opt = {"dt_bias": dev["dt_bias"], "state": dev["state"], "normalize": normalize, "softplus": softplus, "scale": scale,
           "lengths": None if lengths is None else torch.tensor(lengths, device="cuda")}
    god = go.cuda() if layout == "contig" else torch.cat([go, go], -1).cuda()[..., :V]
    announce(f"delta S={S} B={B} H={H} G={G} K={K} V={V} {dtype} {lengths} {layout}")
    dirty()
    out, fs, saved = mdc.delta_forward(*ins, **opt, return_state=True, return_saved=True)
    torch.cuda.synchronize()
    e = slack(S)
    ref.norm_close(out, r["out"], e + (12 * 2.0 ** -12 if dtype == "bf16" else 0.0), "out")
    ref.norm_close(fs, r["state"], e, "state", mag=faded(r["state"], v["state"], e))
    alone, fs2 = mdc.delta_forward(*ins, **opt, return_state=True)
    assert torch.equal(alone, out) and torch.equal(fs2, fs), "without what the backward needs"
    announce("delta backward")
    gr = mdc.delta_backward(god, *ins, saved, **opt, gradFinalState=None if gf is None else gf.cuda())
    torch.cuda.synchronize()
    for name, got in (("gq", gr.q), ("gk", gr.k), ("gv", gr.v), ("gdt", gr.dt), ("gb", gr.b), ("gstate", gr.state)):
        if got is not None:
            mag = r[name + "_before"].norm() if name in ("gq", "gk") else faded(r[name], gf, e) if name == "gstate" else None
            ref.norm_close(got, r[name], e, name, mag=mag)
    ref.norm_close(gr.A, r["gA"], e, "gA", mag=(r["glog"] * r["steps"]).norm())
    if gr.dt_bias is not None:
        ref.norm_close(gr.dt_bias, r["gdt_bias"], e, "gdt_bias", mag=(r["glog"] * r["steps"] * v["A"].abs()).norm() + r["gdt_bias"].norm())
    return ins, opt, god, gf, saved, out, gr


@pytest.mark.parametrize("S,B,H,G,K,V,dtype,lengths,layout,parts", [
    (1, 1, 1, 1, 1, 1, "bf16", None, "contig", {}),
    (1, 2, 4, 2, 128, 256, "fp16", None, "parts", {"state": False}),
    (2, 3, 2, 1, 16, 24, "fp16", [2, 0, 1], "contig", {}),
    (31, 1, 3, 3, 33, 17, "bf16", None, "parts", {}),
    (64, 2, 2, 2, 64, 64, "bf16", None, "contig", {}),
    (65, 2, 4, 1, 65, 80, "fp16", [65, 64], "batch_first", {}),
    (63, 1, 2, 2, 128, 128, "bf16", None, "contig", {"bias": False}),
    (130, 2, 3, 1, 96, 40, "fp16", [33, 130], "parts", {"normalize": False}),
    (129, 1, 2, 1, 128, 65, "bf16", None, "contig", {"softplus": False, "state": False}),
    (70, 1, 1, 1, 7, 130, "bf16", None, "contig", {"scale": -0.7}),
])
def test_against_64_bits(S, B, H, G, K, V, dtype, lengths, layout, parts):
    check(S, B, H, G, K, V, dtype, lengths, layout, seed=S + K, **parts)


@pytest.mark.parametrize("S,B,H,G,K,V,dtype,lengths", [
    (700, 1, 2, 1, 64, 48, "fp16", None),
    (523, 2, 2, 2, 40, 72, "bf16", [300, 523]),
    (400, 3, 1, 1, 128, 16, "fp16", [0, 399, 64]),
])
def test_many_chunks(S, B, H, G, K, V, dtype, lengths):
    check(S, B, H, G, K, V, dtype, lengths, seed=S)


@pytest.mark.parametrize("S,B,H,G,K,V,dtype,lengths,layout", [
    (1300, 1, 2, 1, 64, 48, "fp16", None, "contig"),
    (1250, 2, 1, 1, 100, 130, "bf16", [1250, 70], "parts"),
    (1100, 3, 2, 2, 128, 32, "fp16", [0, 1100, 513], "batch_first"),
])
def test_long_sequences_of_few_heads(S, B, H, G, K, V, dtype, lengths, layout):
    """Cut into segments, whose states before them come from a pass of their own. A state goes through one more
    product for each of up to 16 segments, of the same error as a chunk's: within the bound of S's chunks."""
    check(S, B, H, G, K, V, dtype, lengths, layout, seed=S)


def test_long_sequences_of_rows_that_overlap():
    v, go, _ = inputs(1111, 1, 2, 1, 128, 40, "bf16", 6)
    d = {n: None if t is None else t.cuda() for n, t in v.items()}
    x = torch.randn(1111 * 8 + 80).bfloat16().cuda().as_strided((1111, 1, 2, 40), (8, 8, 40, 1))
    got = [mdc.delta_forward(d["q"], d["k"], y, d["dt"], d["b"], d["A"], dt_bias=d["dt_bias"], state=d["state"],
                             return_state=True) for y in (x, x.contiguous())]
    assert all(torch.equal(p, q) for p, q in zip(*got))


@pytest.mark.parametrize("B,K,dtype", [(35, 128, "bf16"), (40, 64, "fp16")])
def test_more_heads_than_blocks_of_two_waves(B, K, dtype):
    check(130, B, 2, 1, K, 128, dtype, [130] * (B - 5) + [0, 1, 64, 65, 129], "parts", seed=41)


def test_tensors_of_more_than_2_31_values():
    """The last rows, against a call for them alone from the state before them."""
    S, B, H, G, K, V, tail = 64 * 2190, 1, 64, 1, 16, 256, 192
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    q, k, v, dt, b, go = r(S, B, G, K), r(S, B, G, K), r(S, B, H, V), r(S, B, H), r(S, B, H), r(S, B, H, V)
    assert v.numel() > 1 << 31
    A = -torch.rand(H, generator=g, device="cuda")
    announce("delta, more than 2^31 values")
    _, before = mdc.delta_forward(*(t[:S - tail] for t in (q, k, v, dt, b)), A, return_state=True)
    out, end, saved = mdc.delta_forward(q, k, v, dt, b, A, return_state=True, return_saved=True)
    gr = mdc.delta_backward(go, q, k, v, dt, b, A, saved)
    part = [t[S - tail:].clone() for t in (q, k, v, dt, b)]
    out2, end2, saved2 = mdc.delta_forward(*part, A, state=before, return_state=True, return_saved=True)
    gr2 = mdc.delta_backward(go[S - tail:].clone(), *part, A, saved2, state=before)
    torch.cuda.synchronize()
    assert torch.equal(out[S - tail:], out2) and torch.equal(end, end2)
    for name in ("q", "k", "v", "dt", "b"):
        assert torch.equal(getattr(gr, name)[S - tail:], getattr(gr2, name)), name


def test_no_rows():
    s = torch.randn((2, 4, 16, 24), device="cuda")
    dt = torch.bfloat16
    q, v, d = (torch.empty(n, dtype=dt, device="cuda") for n in ((0, 2, 2, 16), (0, 2, 4, 24), (0, 2, 4)))
    A = -torch.ones(4, device="cuda")
    out, fs, saved = mdc.delta_forward(q, q, v, d, d, A, state=s, return_state=True, return_saved=True)
    assert out.shape == (0, 2, 4, 24) and torch.equal(fs, s)
    gf = torch.randn_like(s)
    g = mdc.delta_backward(v, q, q, v, d, d, A, saved, dt_bias=A, state=s, gradFinalState=gf)
    assert torch.equal(g.state, gf) and not g.A.any() and not g.dt_bias.any()


def test_no_length():
    """Every sequence ends before its first row."""
    v, go, gf = inputs(70, 2, 2, 1, 16, 24, "bf16", 3)
    d = {k: t.cuda() for k, t in v.items()}
    ins = (d["q"], d["k"], d["v"], d["dt"], d["b"], d["A"])
    opt = {"dt_bias": d["dt_bias"], "state": d["state"], "lengths": torch.tensor([0, -3], device="cuda")}
    out, fs, saved = mdc.delta_forward(*ins, **opt, return_state=True, return_saved=True)
    g = mdc.delta_backward(go.cuda(), *ins, saved, **opt, gradFinalState=gf.cuda())
    assert not out.any() and torch.equal(fs, d["state"]) and torch.equal(g.state, gf.cuda())
    assert not any(t.any() for t in (g.q, g.k, g.v, g.dt, g.b, g.A, g.dt_bias))


@pytest.mark.parametrize("H,G,K,V,dtype", [(2, 1, 7, 5, "bf16"), (4, 2, 128, 128, "fp16"), (3, 3, 65, 36, "bf16")])
def test_tokens_continue_a_prompt(H, G, K, V, dtype):
    """A prompt cut in two and single tokens against the 64-bit form of the whole."""
    S, B = 81, 3
    v, _, _ = inputs(S, B, H, G, K, V, dtype, seed=K)
    r = ref.delta(v["q"], v["k"], v["v"], v["dt"], v["b"], v["A"], v["dt_bias"], state=v["state"])
    d = {k: t.cuda() for k, t in v.items()}
    announce(f"delta tokens H={H} K={K} V={V}")

    def rows(a, b):
        return tuple(d[n][a:b] for n in ("q", "k", "v", "dt", "b")) + (d["A"],)

    o0, st = mdc.delta_forward(*rows(0, 66), dt_bias=d["dt_bias"], state=d["state"], return_state=True)
    o1, st = mdc.delta_forward(*rows(66, 70), dt_bias=d["dt_bias"], state=st, return_state=True)
    parts = [o0, o1]
    for t in range(70, S):
        *ins, A = rows(t, t + 1)
        parts.append(mdc.delta_step(st, *(x[0] for x in ins), A, dt_bias=d["dt_bias"])[None])
    ref.norm_close(torch.cat(parts), r["out"], slack(S) + (12 * 2.0 ** -12 if dtype == "bf16" else 0), "out")
    ref.norm_close(st, r["state"], slack(S), "state")


def test_token_with_its_options():
    for normalize, softplus in ((False, True), (True, False)):
        v, _, _ = inputs(1, 5, 6, 2, 24, 34, "fp16", seed=9, unit=normalize)
        v["dt"] = v["dt"].abs()
        r = ref.delta(v["q"], v["k"], v["v"], v["dt"], v["b"], v["A"], None, softplus, normalize, 0.3, None, v["state"])
        d = {k: t.cuda() for k, t in v.items()}
        wide = torch.cat([d["v"][0], d["v"][0]], -1)[..., :34]  # rows further apart than they are long
        out = mdc.delta_step(d["state"], d["q"][0], d["k"][0], wide, d["dt"][0], d["b"][0], d["A"], softplus=softplus,
                             normalize=normalize, scale=0.3)
        ref.norm_close(out, r["out"][0], 2.0 ** -18, "out")
        ref.norm_close(d["state"], r["state"], 2.0 ** -18, "state")


def test_rows_apart_and_repeated():
    """Rows of v and gradOut that are one row (stride 0), overlap, or lie too far apart for one buffer."""
    S, B, H, G, K, V = 67, 1, 2, 1, 16, 24
    v, go, _ = inputs(S, B, H, G, K, V, "fp16", seed=5, state=False)
    d = {k: None if t is None else t.cuda() for k, t in v.items()}
    far = torch.zeros((S - 1) * (1 << 24) + H * V, dtype=torch.float16, device="cuda")
    views = {"one": d["v"][:1].expand(S, B, H, V), "overlap": torch.randn(S * 8 + H * V).half().cuda().as_strided((S, B, H, V), (8, 8, V, 1)),
             "far": far.as_strided((S, B, H, V), (1 << 24, H * V, V, 1)).copy_(d["v"])}
    for name, x in views.items():
        announce(f"rows of v: {name}")
        ins = [(d["q"], d["k"], y, d["dt"], d["b"], d["A"]) for y in (x, x.contiguous())]
        (o0, s0), (o1, s1) = (mdc.delta_forward(*i, return_saved=True) for i in ins)
        assert torch.equal(o0, o1), name
        g0 = mdc.delta_backward(x, *ins[0], s0)
        g1 = mdc.delta_backward(x.contiguous(), *ins[1], s1)
        assert all(p is None or torch.equal(p, q) for p, q in zip(g0, g1)), name


def test_decays_at_their_ends():
    """Step sizes from 0 (dt of -infinity) to 300 and rates to -infinity: decays from 1 to 0, and a reset in between."""
    def change(v, go):
        v["dt"][:, 0, 0] = float("-inf")
        v["dt"][::7, 0, 1] = 60.0
        v["dt"][:, 0, 2] = torch.linspace(-14, 40, v["dt"].shape[0]).to(v["dt"].dtype)

    check(100, 1, 4, 2, 32, 40, "fp16", seed=12, change=change)
    v, go, gf = inputs(70, 1, 2, 2, 16, 16, "bf16", 13)
    v["A"][0] = float("-inf")  # every row forgets all before it
    d = {k: t.cuda() for k, t in v.items()}
    ins = (d["q"], d["k"], d["v"], d["dt"], d["b"], d["A"])
    opt = {"dt_bias": d["dt_bias"], "state": d["state"]}
    out, fs, saved = mdc.delta_forward(*ins, **opt, return_state=True, return_saved=True)
    v["A"][0] = -1e4
    r = ref.delta(v["q"], v["k"], v["v"], v["dt"], v["b"], v["A"], v["dt_bias"], state=v["state"], gout=go, gfinal=gf)
    ref.norm_close(out, r["out"], slack(70) + 12 * 2.0 ** -12, "out")
    ref.norm_close(fs, r["state"], slack(70), "state")
    g = mdc.delta_backward(go.cuda(), *ins, saved, **opt, gradFinalState=gf.cuda())
    for name, got in (("gv", g.v), ("gb", g.b)):
        ref.norm_close(got, r[name], slack(70), name)
    for name, got in (("gq", g.q), ("gk", g.k)):
        ref.norm_close(got, r[name], slack(70), name, mag=r[name + "_before"].norm())
    assert torch.isfinite(g.dt).all() and torch.isfinite(g.A).all()


def test_same_keys_and_no_keys():
    """Keys that are all one (the triangular system at its worst), and rows of zeros."""
    def same(v, go):
        v["k"][:] = v["k"][:1]
        v["b"][:] = 4.0

    def none(v, go):
        v["k"][3:40:3] = 0
        v["q"][5:30:5] = 0

    check(128, 1, 2, 1, 32, 32, "fp16", seed=21, change=same)
    check(90, 1, 2, 1, 48, 32, "bf16", seed=22, change=none)


@pytest.mark.parametrize("power", [-90, 90])
def test_sizes_far_from_one(power):
    """Values, states and keys of sizes that fp16 does not have."""
    def change(v, go):
        v["v"].mul_(2.0 ** power)
        v["state"].mul_(2.0 ** power)
        v["k"].mul_(2.0 ** (power // 3))
        v["q"].mul_(2.0 ** (-power // 3))
        go.mul_(2.0 ** -power)

    # |k|^2 + 1e-6 is 1e-6 for the small ones: keys are then near zero, and gradients through them large
    check(70, 1, 2, 1, 32, 32, "bf16", seed=31, change=change, **({"normalize": True}))


def test_what_is_not_finite_stays_in_its_sequence():
    """And, of the rows before it, in its chunk of 64: zeros of the triangular matrices meet it there."""
    v, _, _ = inputs(70, 2, 2, 1, 16, 16, "bf16", 4, state=False)
    v["v"][5, 0, 1, 3] = float("inf")
    v["k"][9, 0] = float("nan")
    d = {k: None if t is None else t.cuda() for k, t in v.items()}
    out, fs = mdc.delta_forward(d["q"], d["k"], d["v"], d["dt"], d["b"], d["A"], return_state=True)
    assert torch.isfinite(out[:, 1]).all() and torch.isfinite(fs[1]).all()
    assert not torch.isfinite(out[20:, 0]).any() and not torch.isfinite(fs[0]).any()
    v, _, _ = inputs(200, 1, 2, 1, 16, 16, "bf16", 4, state=False)
    v["v"][130, 0, 1, 3] = float("inf")
    d = {k: None if t is None else t.cuda() for k, t in v.items()}
    out = mdc.delta_forward(d["q"], d["k"], d["v"], d["dt"], d["b"], d["A"])
    assert torch.isfinite(out[:128]).all() and not torch.isfinite(out[130:, 0, 1, 3]).any()
    assert torch.isfinite(out[:, :, 0]).all() and torch.isfinite(out[:, 0, 1, :3]).all()


def test_same_bits_again():
    ins, opt, god, gf, saved, out, gr = check(200, 2, 4, 2, 64, 64, "bf16", [200, 131], "parts", seed=8)
    dirty()
    out2, saved2 = mdc.delta_forward(*ins, **opt, return_saved=True)
    g2 = mdc.delta_backward(god, *ins, saved2, **opt, gradFinalState=gf.cuda())
    assert torch.equal(out, out2)
    assert all(p is None or torch.equal(p, q) for p, q in zip(gr, g2))


def test_larger_than_one_block_a_die():
    """More heads than compute units, on the device against a float64 walk over chunks of one row."""
    S, B, H, G, K, V = 130, 40, 8, 8, 64, 64
    v, _, _ = inputs(S, B, H, G, K, V, "bf16", 2, state=False)
    d = {k: None if t is None else t.cuda() for k, t in v.items()}
    out, fs = mdc.delta_forward(d["q"], d["k"], d["v"], d["dt"], d["b"], d["A"], dt_bias=d["dt_bias"], return_state=True)
    s = torch.zeros((B, H, K, V), dtype=torch.float64, device="cuda")
    want = []
    for t in range(S):
        kn, qn = (ref.unit(d[n][t].double(), True) for n in ("k", "q"))
        s = s * torch.exp(d["A"].double() * torch.nn.functional.softplus(d["dt"][t].double() + d["dt_bias"].double()))[..., None, None]
        u = torch.sigmoid(d["b"][t].double())[..., None] * (d["v"][t].double() - (kn[..., None] * s).sum(-2))
        s = s + kn[..., None] * u[..., None, :]
        want.append((qn[..., None] * s).sum(-2) * K ** -0.5)
    ref.norm_close(out, torch.stack(want).cpu(), slack(S) + 12 * 2.0 ** -12, "out")
    ref.norm_close(fs, s.cpu(), slack(S), "state")
