"""Selective state space scan against the 64-bit form.

Tolerances, relative to the sums of absolute terms (mag). A row's step size has a relative error
under 2^-21 (softplus in fp32), its decay exp(d A) one under 2^-21 (|d A| + 1), and each state update
two roundings; decays do not grow anything, so after T rows a state is within
T 2^-21 (2 + max |d A|) of mag, and the inputs here keep |d A| under 6: T 2^-18 as a bound that no
rounding pattern reaches. Outputs and gradients add sums of at most 32 states and 16 rows in fp32 and
a gradient's own recurrence of T rows: (2 T + 64) 2^-18 in all. Sums over channels are fp32 sums of
at most 64 terms and then of the blocks: under the same 64."""
from __future__ import annotations

import pytest
import torch

import masked_depthwise_causal_amd as mdc

from . import ssm_ref as ref
from .gpu_util import announce
from .test_conv_act import DT, dirty, lay, rand

pytestmark = pytest.mark.gpu


def slack(T):
    return (2 * T + 64) * 2.0 ** -18


def inputs(S, B, H, N, G, dtype, seed, gate=True, skip=True, bias=True, state=True):
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    v = {"x": rand(g, S, B, H, dt=dt), "dt": rand(g, S, B, H, dt=dt, scale=0.5),
         "A": -torch.rand((N, H), generator=g) * 3 - 0.05,
         "Bm": rand(g, S, B, G, N, dt=dt), "Cm": rand(g, S, B, G, N, dt=dt),
         "D": torch.randn(H, generator=g) if skip else None,
         "z": rand(g, S, B, H, dt=dt) if gate else None,
         "dt_bias": torch.randn(H, generator=g) - 2 if bias else None,
         "state": torch.randn((B, N, H), generator=g) if state else None}
    return v, rand(g, S, B, H, dt=dt), torch.randn((B, N, H), generator=g) if state else None


def check(S, B, H, N, G, dtype, lengths=None, layout="contig", softplus=True, seed=0, **parts):
    v, go, gf = inputs(S, B, H, N, G, dtype, seed, **parts)
    if not softplus:  # dt and its bias are then the step size itself, which is positive
        v["dt"], v["dt_bias"] = v["dt"].abs(), None if v["dt_bias"] is None else v["dt_bias"].abs()
    r = ref.scan(v["x"], v["dt"], v["A"], v["Bm"], v["Cm"], v["D"], v["z"], v["dt_bias"], softplus,
                 lengths, v["state"], go, gf)
    for b, n in enumerate(ref.lens_of(lengths, S, B)):  # what dead rows hold must not matter
        for k in ("x", "dt", "Bm", "Cm", "z"):
            if v[k] is not None:
                v[k][n:, b] = float("nan")
        go[n:, b] = float("inf")
    dev = {k: None if t is None else t.cuda() for k, t in v.items()}
    for k in ("x", "dt", "z"):
        if v[k] is not None:
            dev[k] = lay(v[k], layout)
    if layout != "contig":  # B and C as parts of one projection's rows
        both = torch.cat([v["Bm"], v["Cm"]], -1).cuda()
        dev["Bm"], dev["Cm"] = both[..., :N], both[..., N:]
    ins = tuple(dev[k] for k in ("x", "dt", "A", "Bm", "Cm"))
    opt = {k: dev[k] for k in ("D", "z", "dt_bias", "state")}
    opt |= {"softplus": softplus,
            "lengths": None if lengths is None else torch.tensor(lengths, device="cuda")}
    announce(f"scan S={S} B={B} H={H} N={N} G={G} {dtype} {lengths} {layout}")
    dirty()
    out, fs, saved = mdc.scan_forward(*ins, **opt, return_state=True, return_saved=True)
    god, gfd = lay(go, layout), None if gf is None else gf.cuda()
    torch.cuda.synchronize()
    e = slack(S)
    ref.close(out, r["out"], e, "out")
    ref.close(fs, r["state"], e, "state")
    announce("scan backward")
    gr = mdc.scan_backward(god, *ins, saved, **opt, gradFinalState=gfd)
    torch.cuda.synchronize()
    for name, got, key in (("gx", gr.x, "gx"), ("gdt", gr.dt, "gdt"), ("gA", gr.A, "gA"),
                           ("gB", gr.B, "gB"), ("gC", gr.C, "gC"), ("gD", gr.D, "gD"),
                           ("gz", gr.z, "gz"), ("gdt_bias", gr.dt_bias, "gbias"),
                           ("gstate", gr.state, "gs")):
        if got is not None:
            ref.close(got, r[key], e, name)
    return ins, opt, god, gfd, saved, out, gr


@pytest.mark.parametrize("S,B,H,N,G,dtype,lengths,layout,parts", [
    (1, 1, 1, 1, 1, "bf16", None, "contig", {}),
    (2, 2, 64, 16, 1, "fp16", None, "contig", {}),
    (15, 1, 65, 4, 1, "bf16", None, "contig", {"gate": False}),
    (16, 3, 63, 5, 1, "fp16", [16, 0, 1], "slice", {}),
    (17, 2, 130, 8, 2, "bf16", None, "batch_first", {"skip": False}),
    (40, 2, 96, 16, 3, "fp16", [33, 40], "contig", {"bias": False}),
    (33, 1, 70, 17, 1, "bf16", None, "channels_apart", {"state": False}),
    (35, 2, 100, 32, 2, "fp16", [32, 35], "slice", {}),
    (19, 1, 12, 3, 4, "bf16", None, "contig", {"softplus": False, "gate": False, "state": False}),
])
def test_against_64_bits(S, B, H, N, G, dtype, lengths, layout, parts):
    check(S, B, H, N, G, dtype, lengths, layout, seed=S + H, **parts)


@pytest.mark.parametrize("S,B,H,N,dtype,lengths", [
    (700, 1, 40, 16, "bf16", None),       # cut into chunks
    (523, 2, 33, 6, "fp16", [300, 523]),  # a sequence that ends in an earlier chunk
    (300, 2, 20, 32, "bf16", [0, 299]),
])
def test_long_sequences_in_chunks(S, B, H, N, dtype, lengths):
    check(S, B, H, N, 1, dtype, lengths, seed=S)


def test_no_rows():
    s = torch.randn((2, 4, 16), device="cuda")
    e = torch.empty((0, 2, 16), dtype=torch.bfloat16, device="cuda")
    c = torch.empty((0, 2, 4), dtype=torch.bfloat16, device="cuda")
    A = -torch.ones((4, 16), device="cuda")
    out, fs, saved = mdc.scan_forward(e, e, A, c, c, state=s, return_state=True, return_saved=True)
    assert out.shape == (0, 2, 16) and torch.equal(fs, s)
    gf = torch.randn_like(s)
    g = mdc.scan_backward(e, e, e, A, c, c, saved, state=s, gradFinalState=gf)
    assert torch.equal(g.state, gf) and not g.A.any()


@pytest.mark.parametrize("H,N,G,dtype", [(7, 3, 1, "bf16"), (130, 16, 2, "fp16"), (64, 32, 1, "bf16")])
def test_tokens_continue_a_prompt(H, N, G, dtype):
    """A prompt cut in two and single tokens against the 64-bit form of the whole."""
    S, B = 21, 3
    v, _, _ = inputs(S, B, H, N, G, dtype, seed=H)
    r = ref.scan(v["x"], v["dt"], v["A"], v["Bm"], v["Cm"], v["D"], v["z"], v["dt_bias"], True, None,
                 v["state"])
    d = {k: t.cuda() for k, t in v.items()}
    announce(f"scan tokens H={H} N={N}")

    def rows(a, b):
        return (d["x"][a:b], d["dt"][a:b], d["A"], d["Bm"][a:b], d["Cm"][a:b])

    def opt(a, b):
        return {"D": d["D"], "z": d["z"][a:b], "dt_bias": d["dt_bias"]}

    o0, st = mdc.scan_forward(*rows(0, 9), **opt(0, 9), state=d["state"], return_state=True)
    o1, st = mdc.scan_forward(*rows(9, 13), **opt(9, 13), state=st, return_state=True)
    parts = [o0, o1]
    for t in range(13, S):
        x, dt, A, Bm, Cm = rows(t, t + 1)
        parts.append(mdc.scan_step(st, x[0], dt[0], A, Bm[0], Cm[0], D=d["D"], z=d["z"][t],
                                   dt_bias=d["dt_bias"])[None])
    ref.close(torch.cat(parts), r["out"], slack(S), "out")
    ref.close(st, r["state"], slack(S), "state")


def test_one_group_without_its_axis():
    v, go, _ = inputs(20, 2, 64, 4, 1, "bf16", seed=1, state=False)
    d = {k: None if t is None else t.cuda() for k, t in v.items()}
    a, sa = mdc.scan_forward(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], return_saved=True)
    b, sb = mdc.scan_forward(d["x"], d["dt"], d["A"], d["Bm"][:, :, 0], d["Cm"][:, :, 0],
                             return_saved=True)
    assert torch.equal(a, b)
    g = mdc.scan_backward(go.cuda(), d["x"], d["dt"], d["A"], d["Bm"][:, :, 0], d["Cm"][:, :, 0], sb)
    assert g.B.shape == (20, 2, 4) and g.C.shape == (20, 2, 4)


def test_large_and_small_step_sizes():
    """Step sizes from 1e-6 (softplus of -14) to 40: the decay goes from 1 - 1e-6 to zero."""
    v, go, gf = inputs(48, 1, 64, 4, 1, "bf16", seed=2)
    v["dt"] = torch.linspace(-14, 40, 48).view(-1, 1, 1).expand(48, 1, 64).bfloat16()
    r = ref.scan(v["x"], v["dt"], v["A"], v["Bm"], v["Cm"], v["D"], v["z"], v["dt_bias"], True, None,
                 v["state"])
    d = {k: t.cuda() for k, t in v.items()}
    out, fs = mdc.scan_forward(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], D=d["D"], z=d["z"],
                               dt_bias=d["dt_bias"], state=d["state"], return_state=True)
    # |d A| reaches 120, so a decay's relative error grows to 120 2^-21: where it does the decay is
    # under exp(-6) of its input, and the bound for |d A| < 6 covers the product
    ref.close(out, r["out"], slack(48), "out")
    ref.close(fs, r["state"], slack(48), "state")


def test_same_bits_again():
    ins, opt, god, gfd, saved, out, gr = check(290, 2, 100, 16, 1, "bf16", [290, 131], "slice", seed=8)
    dirty()
    out2, saved2 = mdc.scan_forward(*ins, **opt, return_saved=True)
    g2 = mdc.scan_backward(god, *ins, saved2, **opt, gradFinalState=gfd)
    assert torch.equal(out, out2)
    assert all(p is None or torch.equal(p, q) for p, q in zip(gr, g2))
