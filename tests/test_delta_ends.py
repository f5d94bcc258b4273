"""Gated delta rule where numbers, gates and lengths reach their ends, against the 64-bit form: outputs next to their own
rounding, rows far smaller than the others, gates that are open or shut, what stands at and past a length.

`slack` is the bound of test_delta.py, relative to a whole tensor's norm. A single row's, or a single gate's, result may be
a small difference of its parts: 16 times as much, as for single values there."""
from __future__ import annotations

import pytest
import torch

import masked_depthwise_causal_amd as mdc

from . import delta_ref as ref
from .gpu_util import announce
from .ssm_ref import F
from .test_conv_act import DT
from .test_delta import inputs, slack

pytestmark = pytest.mark.gpu


def both(v, go, gf=None, lengths=None, **opt):
    """The 64-bit results, the outputs and the gradients."""
    r = ref.delta(v["q"], v["k"], v["v"], v["dt"], v["b"], v["A"], v["dt_bias"], normalize=opt.get("normalize", True),
                  lengths=lengths, state=v["state"], gout=go, gfinal=gf)
    out, end, g = run(v, go, gf, lengths, **opt)
    return r, out, end, g


def run(v, go, gf=None, lengths=None, **opt):
    d = {n: None if t is None else t.cuda() for n, t in v.items()}
    ins = (d["q"], d["k"], d["v"], d["dt"], d["b"], d["A"])
    opt |= {"dt_bias": d["dt_bias"], "state": d["state"],
            "lengths": None if lengths is None else torch.tensor(lengths, device="cuda")}
    out, end, saved = mdc.delta_forward(*ins, **opt, return_state=True, return_saved=True)
    g = mdc.delta_backward(go.cuda(), *ins, saved, **opt, gradFinalState=None if gf is None else gf.cuda())
    torch.cuda.synchronize()
    return out, end, g


def row_near(got, want, size, e, name):
    """One row, or what is compared as one: its rounding, and e of `size`."""
    half = torch.finfo(got.dtype).eps / 2
    got = got.detach().cpu().to(F)
    assert torch.isfinite(got).all(), name
    off, allowed = float((got - want).norm()), float(half * want.norm() + e * size.norm())
    assert off <= allowed, f"{name}: {off} of {float(want.norm())}, {allowed} allowed"


@pytest.mark.parametrize("S,B,H,G,K,V", [(64, 2, 2, 2, 64, 64), (130, 35, 2, 1, 128, 128), (100, 3, 4, 2, 96, 80)])
def test_outputs_in_bf16_are_rounded_once(S, B, H, G, K, V):
    """A value within d of the 64-bit one is another bf16 number than that one's for d of each rounding step, up to 2^-7 of
    it, and then a step off: squares of the differences add up to 2^-7 |v| |d|, or sqrt(2^-7 slack) of the norm."""
    v, go, _ = inputs(S, B, H, G, K, V, "bf16", S + K)
    r = ref.delta(v["q"], v["k"], v["v"], v["dt"], v["b"], v["A"], v["dt_bias"], state=v["state"])
    d = {n: t.cuda() for n, t in v.items()}
    announce(f"bf16 outputs S={S} B={B} K={K}")
    out = mdc.delta_forward(*(d[n] for n in ("q", "k", "v", "dt", "b", "A")), dt_bias=d["dt_bias"], state=d["state"])
    once = r["out"].to(torch.bfloat16).to(F)
    off = float((out.cpu().to(F) - once).norm() / once.norm())
    assert off <= (2.0 ** -7 * slack(S)) ** 0.5, off


def small_rows(power, normalize, dtype="bf16"):
    v, go, gf = inputs(90, 1, 2, 1, 32, 24, dtype, 50, unit=normalize)
    for name, rows in (("k", (20, 70)), ("q", (33, 34, 80))):
        for i in rows:
            v[name][i] *= 2.0 ** power
    v["k"][10] = v["q"][12] = 0
    return v, go, gf


@pytest.mark.parametrize("power,normalize", [(-30, True), (-44, True), (-52, True), (-65, True), (-90, True), (-44, False), (-70, False)])
def test_gradients_of_small_rows(power, normalize):
    """Of q and k, each row next to its own size: they are g / sqrt(1e-6) where normalized, 1000 times the others'."""
    v, go, gf = small_rows(power, normalize)
    announce(f"small rows 2^{power}, normalize={normalize}")
    r, _, _, g = both(v, go, gf, normalize=normalize)
    for name, got in (("gk", g.k), ("gq", g.q)):
        for i in range(90):
            row_near(got[i], r[name][i], r[name + "_before"][i], 16 * slack(90), f"{name} row {i}")


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_rows_of_zeros_beside_others(dtype):
    """Keys and queries of zeros in one chunk, as padding has them: gradients of the other rows; and states of small keys."""
    v, go, gf = inputs(90, 1, 2, 1, 32, 24, dtype, 54)
    v["k"][10:12] = v["q"][11:13] = 0
    announce(f"rows of zeros {dtype}")
    r, _, _, g = both(v, go, gf)
    for name, got in (("gk", g.k), ("gq", g.q)):
        for i in range(90):
            row_near(got[i], r[name][i], r[name + "_before"][i], 16 * slack(90), f"{name} row {i}")
    if dtype == "bf16":
        v, go, _ = inputs(90, 1, 2, 1, 32, 24, dtype, 55, unit=False, state=False)
        v["k"] *= 2.0 ** -30
        v["k"][10:12] = 0
        r, _, end, _ = both(v, go, normalize=False)
        ref.norm_close(end, r["state"], slack(90), "state")


@pytest.mark.parametrize("power,normalize", [(-30, True), (-44, True), (-65, True), (-90, True), (-44, False), (-70, False)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_outputs_of_small_rows(power, normalize, dtype):
    """Of queries, each row next to its own size (in fp16 as small as its numbers are)."""
    if dtype == "fp16":
        power //= 8
    v, go, gf = small_rows(power, normalize, dtype)
    if dtype == "fp16":
        v["v"] *= 64
        v["state"] *= 64
    announce(f"small rows 2^{power} {dtype}, normalize={normalize}")
    r, out, _, _ = both(v, go, gf, normalize=normalize)
    for i in range(90):
        tiny = torch.full_like(r["out"][i], torch.finfo(out.dtype).smallest_normal)  # results below it have fewer bits
        row_near(out[i], r["out"][i], r["out"][i].abs() + tiny / (16 * slack(90)), 16 * slack(90), f"row {i}")


@pytest.mark.parametrize("S,B,H,K,V", [(70, 2, 2, 16, 24), (1100, 3, 2, 32, 24), (1300, 2, 1, 100, 130)])
def test_state_of_sequences_that_ended(S, B, H, K, V):
    """No rows: the state that came in, in all its bits, where the sequence is cut into segments too."""
    v, go, gf = inputs(S, B, H, 1, K, V, "bf16", S)
    lengths = [0, S, -1][:B]
    sizes = torch.arange(K)[None, None, :, None] % 61 - 30.0
    v["state"] *= torch.exp2(sizes)
    v["state"][0, 0, 3, 2] = float("inf")
    v["state"][0, 0, 4, 5] = 2.0 ** -126
    announce(f"ended sequences S={S}")
    out, end, g = run(v, go, gf, lengths)
    for b in range(B):
        if lengths[b] <= 0:
            assert torch.equal(end[b], v["state"][b].cuda()), b
            assert torch.equal(g.state[b], gf[b].cuda()), b
            assert not out[:, b].any()


@pytest.mark.parametrize("B,H,V", [(1, 2, 24), (40, 8, 64)])
@pytest.mark.parametrize("what", ["v", "k", "q", "go"])
def test_rows_past_a_length_beside_rows_that_are_not_finite(B, H, V, what):
    S, n = 130, 70
    v, go, gf = inputs(S, B, H, 1, 16, V, "bf16", 51)
    (go if what == "go" else v[what])[66] = float("inf")
    announce(f"not finite in {what}, B={B}")
    out, _, g = run(v, go, gf, [n] * B)
    for name, t in (("out", out), ("gq", g.q), ("gk", g.k), ("gv", g.v), ("gdt", g.dt), ("gb", g.b)):
        assert not t[n:].any(), name
    assert not torch.isfinite((g.v if what == "go" else out)[66]).all()


@pytest.mark.parametrize("dtype,open_,size", [("bf16", 20, 1.0), ("fp16", 12, 256.0)])
def test_gradients_of_open_and_shut_gates(dtype, open_, size):
    """Each gate's next to the slope of its own logistic function."""
    v, go, gf = inputs(100, 2, 2, 1, 32, 24, dtype, 52)
    u = torch.rand((100, 2), generator=torch.Generator().manual_seed(1))
    v["b"][..., 0], v["b"][..., 1] = (6 + (open_ - 6) * u).to(DT[dtype]), -(6 + 6 * u).to(DT[dtype])
    go, gf = (go.float() * size).to(DT[dtype]), gf * size
    announce(f"open and shut gates, {dtype}")
    r, _, _, g = both(v, go, gf)
    b = v["b"].to(F)
    slope = torch.sigmoid(b) * torch.sigmoid(-b)
    half = torch.finfo(g.b.dtype).eps / 2
    for h in (0, 1):
        want, got = (r["gb"] / slope)[..., h], (g.b.cpu().to(F) / slope)[..., h]
        assert float((got - want).norm()) <= float((half + 16 * slack(100)) * want.norm()), h


def test_tokens_of_large_rows():
    """Keys and queries whose squares are past fp32's largest, next to ordinary and small ones."""
    v, _, _ = inputs(1, 6, 4, 2, 100, 40, "bf16", 53)
    v["k"][0, 1] *= 2.0 ** 70
    v["q"][0, 2] *= 2.0 ** 100
    v["k"][0, 3] *= 2.0 ** 64
    v["q"][0, 3] *= 2.0 ** -70
    v["k"][0, 4, 0, 70:] *= 2.0 ** 90
    r = ref.delta(v["q"], v["k"], v["v"], v["dt"], v["b"], v["A"], v["dt_bias"], state=v["state"])
    d = {n: t.cuda() for n, t in v.items()}
    out = mdc.delta_step(d["state"], *(d[n][0] for n in ("q", "k", "v", "dt", "b")), d["A"], dt_bias=d["dt_bias"])
    for b in range(6):
        row_near(out[b], r["out"][0, b], r["out"][0, b].abs(), 2.0 ** -18, f"out {b}")
        ref.norm_close(d["state"][b], r["state"][b], 2.0 ** -18, f"state {b}")
