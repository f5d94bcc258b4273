"""Infinities, NaN and the types' largest values in live rows of the state space block's operators.

Each case is compared bit for bit with the same call on finite values of the same limit (a step size's
pre-activation of -200 has exp(-200), which is below the smallest fp32 number), and that call with the
64-bit form, to the bounds of the operators' own tests."""
from __future__ import annotations

import pytest
import torch

import masked_depthwise_causal_amd as mdc

from . import ssm_ref as ref
from .gpu_util import announce
from .test_conv_act import DT, GX, dirty, rand
from .test_scan import inputs, slack

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def same(a, b, name):
    """Equal bits, NaN equal to NaN."""
    assert a.shape == b.shape and a.dtype == b.dtype, name
    ok = (a == b) | (torch.isnan(a) & torch.isnan(b))
    assert bool(ok.all()), f"{name}: {int((~ok).sum())} of {ok.numel()} differ"


def scan_both(v, go, gf, lengths=None):
    """Everything that the scan's forward and backward give for the inputs `v`, by name."""
    d = {k: None if t is None else t.cuda() for k, t in v.items()}
    ins = tuple(d[k] for k in ("x", "dt", "A", "Bm", "Cm"))
    opt = {k: d[k] for k in ("D", "z", "dt_bias", "state")}
    opt["lengths"] = None if lengths is None else torch.tensor(lengths, device="cuda")
    dirty()
    out, fs, saved = mdc.scan_forward(*ins, **opt, return_state=True, return_saved=True)
    gr = mdc.scan_backward(go.cuda(), *ins, saved, **opt, gradFinalState=gf.cuda())
    torch.cuda.synchronize()
    return {"out": out, "state": fs, "gx": gr.x, "gdt": gr.dt, "gA": gr.A, "gB": gr.B, "gC": gr.C,
            "gD": gr.D, "gz": gr.z, "gbias": gr.dt_bias, "gs": gr.state}


def against_64_bits(got, v, go, gf, S, lengths=None):
    r = ref.scan(v["x"], v["dt"], v["A"], v["Bm"], v["Cm"], v["D"], v["z"], v["dt_bias"], True, lengths,
                 v["state"], go, gf)
    for k, t in got.items():
        ref.close(t, r[k], slack(S), k)


@pytest.mark.parametrize("S,H,N,dtype", [(37, 70, 16, "bf16"), (20, 64, 8, "fp16"), (40, 33, 32, "bf16"),
                                         (600, 40, 16, "bf16")])  # the last one is cut into chunks
def test_step_of_minus_infinity_leaves_the_state_alone(S, H, N, dtype):
    v, go, gf = inputs(S, 2, H, N, 1, dtype, seed=S)
    rows = torch.rand((S, 2, H), generator=torch.Generator().manual_seed(1)) < 0.3
    rows[S // 2] = True  # a whole row
    v["dt"][rows] = -200.0
    v["dt_bias"][3] = -200.0  # a whole channel
    announce(f"scan, steps of -200 S={S} H={H} N={N}")
    want = scan_both(v, go, gf)
    against_64_bits(want, v, go, gf, S)
    w = dict(v, dt=v["dt"].clone(), dt_bias=v["dt_bias"].clone())
    w["dt"][rows] = -INF
    w["dt_bias"][3] = -INF
    announce(f"scan, steps of -inf S={S} H={H} N={N}")
    got = scan_both(w, go, gf)
    for k in want:
        same(got[k], want[k], k)
    assert not got["gdt"][rows.cuda()].any()


@pytest.mark.parametrize("N,dtype", [(16, "bf16"), (5, "fp16")])
def test_token_of_minus_infinity_leaves_the_state_alone(N, dtype):
    v, _, _ = inputs(1, 3, 70, N, 1, dtype, seed=N)
    d = {k: t.cuda() for k, t in v.items()}
    d["dt"][0, 1] = -INF
    st = d["state"].clone()
    out = mdc.scan_step(st, d["x"][0], d["dt"][0], d["A"], d["Bm"][0], d["Cm"][0], D=d["D"], z=d["z"][0],
                        dt_bias=d["dt_bias"])
    assert torch.equal(st[1], d["state"][1])
    v["dt"][0, 1] = -200.0
    r = ref.scan(v["x"], v["dt"], v["A"], v["Bm"], v["Cm"], v["D"], v["z"], v["dt_bias"], True, None,
                 v["state"])
    ref.close(out[None], r["out"], slack(1), "out")


@pytest.mark.parametrize("value", [INF, NAN])
def test_other_channels_do_not_see_a_step_that_is_not_finite(value):
    S, H = 37, 70
    v, go, gf = inputs(S, 2, H, 16, 1, "bf16", seed=4)
    want = scan_both(v, go, gf)
    w = dict(v, dt=v["dt"].clone())
    w["dt"][S // 2, 0, 5] = value
    got = scan_both(w, go, gf)
    others = torch.arange(H, device="cuda") != 5
    for k in ("out", "state", "gx", "gdt", "gA", "gD", "gz", "gbias", "gs"):
        same(got[k][..., others], want[k][..., others], k)
    same(got["out"][:S // 2, 0, 5], want["out"][:S // 2, 0, 5], "rows before")
    assert not torch.isfinite(got["out"][S // 2:, 0, 5]).any()
    same(got["out"][:, 1], want["out"][:, 1], "the other sequence")


@pytest.mark.parametrize("M,N", [(3, 40), (130, 72)])  # few rows and tiles
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_softplus_epilogue_at_the_ends(M, N, dtype):
    dt = DT[dtype]
    big = torch.finfo(dt).max
    ends = [-INF, -big, -200.0, -20.0, 0.0, 20.0, big / 2, big, INF, NAN]
    bias = torch.tensor([ends[i % len(ends)] for i in range(N)]).to(dt)
    g = torch.Generator().manual_seed(M)
    x, w = torch.randn((M, 64), generator=g).to(dt), torch.randn((N, 64), generator=g).to(dt) * 0.1
    w[6::len(ends)] = w[7::len(ends)] = 0  # sums beyond the type are another matter
    pre = x.to(ref.F) @ w.to(ref.F).t() + bias.to(ref.F)
    mag = x.to(ref.F).abs() @ w.to(ref.F).abs().t() + bias.to(ref.F).abs()
    want = ref.softplus(pre)
    # an error of pre counts by the slope there, and softplus has a relative error of its own
    mag = torch.nan_to_num(mag * ref.sigmoid(pre), nan=0.0) + want
    announce(f"linear softplus ends M={M} N={N} {dtype}")
    got = mdc.linear_forward(x.cuda(), w.cuda(), bias.cuda(), activation="softplus").cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[torch.isinf(want)].to(ref.F), want[torch.isinf(want)])
    fine = torch.isfinite(want)
    ref.close(got[fine], (want[fine], mag[fine]), (64 + 64) * 2.0 ** -23, "softplus")


@pytest.mark.parametrize("S,H,W,lengths", [(37, 20, 4, [37, 0, 30]), (11, 7, 3, [11, 1, 8]),
                                           (70, 133, 2, [64, 70, 63]), (9, 64, 1, [9, 4, 0])])
@pytest.mark.parametrize("value", [INF, -INF, NAN])
def test_conv_rows_past_a_length_do_not_meet_the_weights(S, H, W, lengths, value):
    """Zeros there, and nothing of them in the last rows before the length, for weights that make
    something else of a product with zero."""
    g = torch.Generator().manual_seed(S)
    x, gy, w = rand(g, S, 3, H), rand(g, S, 3, H), rand(g, W, H)
    state, gf = rand(g, W - 1, 3, H), rand(g, W - 1, 3, H)
    for k in range(W):
        w[k, k::7] = value
    r = ref.conv(x, w, None, None, lengths, state, gy, gf)
    n = torch.tensor(lengths, device="cuda")
    announce(f"conv weights of {value} S={S} H={H} W={W}")
    dirty()
    gr = mdc.conv_act_backward(gy.cuda(), x.cuda(), w.cuda(), activation=None, lengths=n,
                               state=state.cuda(), gradFinalState=gf.cuda())
    for b, m in enumerate(lengths):
        assert not gr.x[m:, b].any(), "rows past the length"
    for got, key in ((gr.x, "gx"), (gr.state, "gs")):
        got, (want, mag) = got.cpu(), r[key]
        fine = torch.isfinite(want)
        same(torch.where(fine, torch.zeros((), dtype=ref.F), got.to(ref.F)),
             torch.where(fine, torch.zeros((), dtype=ref.F), want), key)
        ref.close(got[fine], (want[fine], mag[fine]), GX, key)


@pytest.mark.parametrize("S,H,N,dtype,lengths", [(37, 70, 16, "bf16", None), (16, 64, 8, "fp16", [16, 3]),
                                                 (600, 40, 16, "bf16", [600, 290])])  # in chunks
def test_rates_of_minus_infinity_forget_the_state(S, H, N, dtype, lengths):
    """The decay is 0 then, and 1 in rows past the length, which leave the state alone."""
    v, go, gf = inputs(S, 2, H, N, 1, dtype, seed=S)
    rates = torch.rand((N, H), generator=torch.Generator().manual_seed(2)) < 0.3
    v["A"][rates] = -1e30
    announce(f"scan, rates of -1e30 S={S} H={H} N={N}")
    want = scan_both(v, go, gf, lengths)
    against_64_bits(want, v, go, gf, S, lengths)
    for value in (-3e38, -INF):
        announce(f"scan, rates of {value} S={S} H={H} N={N}")
        got = scan_both(dict(v, A=torch.where(rates, value, v["A"])), go, gf, lengths)
        for k in want:
            same(got[k], want[k], k)


def test_token_with_rates_of_minus_infinity():
    v, _, _ = inputs(1, 3, 70, 5, 1, "bf16", seed=6)
    d = {k: t.cuda() for k, t in v.items()}
    d["dt"][0, 0] = -INF  # no step: the state stays, whatever the rate
    res = []
    for value in (-1e30, -INF):
        A, st = d["A"].clone(), d["state"].clone()
        A[2] = value
        out = mdc.scan_step(st, d["x"][0], d["dt"][0], A, d["Bm"][0], d["Cm"][0], D=d["D"], z=d["z"][0],
                            dt_bias=d["dt_bias"])
        res.append((out, st))
    same(res[1][0], res[0][0], "out")
    same(res[1][1], res[0][1], "state")
    assert torch.equal(res[1][1][0], d["state"][0])


@pytest.mark.parametrize("act", ["silu", "gelu", "relu", "softplus"])
@pytest.mark.parametrize("dtype,big", [("fp16", 65504.0), ("bf16", 1e20), ("bf16", 3.3895313892515355e38)])
@pytest.mark.parametrize("M", [5, 100])
def test_slopes_of_large_and_infinite_values(act, dtype, big, M):
    """Slopes are 0 and 1 at the ends; pre is infinite where its sum is beyond a 16-bit type."""
    dt, N, K = DT[dtype], 48, 40
    g = torch.Generator().manual_seed(M)
    x, w, go = (torch.randn(s, generator=g).to(dt) for s in ((M, K), (N, K), (M, N)))
    pre = torch.randn((M, N), generator=g).to(dt)
    p64 = pre.to(ref.F)
    for i, v in enumerate((big, -big, INF, -INF, 300.0, -300.0)):
        pre[:, i::8] = v
        p64[:, i::8] = max(min(v, 1e5), -1e5)  # whose slopes are 0 and 1 in 64 bits
    announce(f"linear slopes {act} {dtype} {big} M={M}")
    gr = mdc.linear_backward(go.cuda(), x.cuda(), w.cuda(), pre.cuda(), activation=act)
    slope = ref.act_slope(p64, act)
    gg = go.to(ref.F) * slope
    gm = go.to(ref.F).abs() * (slope.abs() + 2.0 ** -10 * (1 + p64.abs().clamp(max=4)))
    half = torch.finfo(dt).eps / 2
    e = lambda K: (K + 64) * 2.0 ** -23  # noqa: E731  as in test_linear.py
    ref.close(gr.x, (gg @ w.to(ref.F), gm @ w.to(ref.F).abs()), half + e(N), "gx")
    ref.close(gr.weight, (gg.t() @ x.to(ref.F), gm.t() @ x.to(ref.F).abs()), half + e(M), "gw")
    ref.close(gr.bias, (gg.sum(0), gm.sum(0)), e(M), "gbias")


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradients_where_pre_is_beyond_fp16(act):
    """The forward's sums are fp32, and its output is finite where pre is far below the type's range."""
    g = torch.Generator().manual_seed(1)
    x, w, go = (torch.randn(s, generator=g).half() for s in ((70, 64), (40, 64), (70, 40)))
    x[:, 0], w[::2, 0] = 300.0, -300.0  # pre near -90000 in every other column
    out, pre = mdc.linear_forward(x.cuda(), w.cuda(), activation=act, return_pre=True)
    assert not out[:, ::2].any() and torch.isinf(pre[:, ::2]).all()
    gr = mdc.linear_backward(go.cuda(), x.cuda(), w.cuda(), pre, activation=act)
    assert all(torch.isfinite(t).all() for t in gr)
    assert not gr.weight[::2].any() and not gr.bias[::2].any()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_gates_slope_at_large_values(dtype):
    """gz where the gate is large, up to the type's largest value and infinity."""
    S, H, big = 20, 64, torch.finfo(DT[dtype]).max
    v, go, gf = inputs(S, 1, H, 16, 1, dtype, seed=3)
    v["z"][:, :, 0], v["z"][:, :, 1] = -big, -300.0
    got = scan_both(v, go, gf)
    assert not got["gz"][:, :, :2].any() and not got["out"][:, :, :2].any()
    v["z"][:, :, 0] = INF  # a slope of 1
    assert bool(torch.isfinite(scan_both(v, go, gf)["gz"]).all())
