"""The product's gradients against the chain without roundings in between: pre in 64 bits, its slope, and
the sums. What lies between is bounded by itself: pre's rounding (to 16 bits or fp32) times the slope's
own largest slope, and g's rounding to 16 bits, which gbias does not see.

    |pre - exact| <= (K + 64) 2^-23 mag (its fp32 sum) + half a step of |pre|            =: dp
    |slope - exact| <= max |act''| dp + 2^-21 (1 + |pre|) (fp32 functions)
    gbias: |gout| times that over the rows, and an fp32 sum; gx and gw: as much of |w|, |x|, and half a
    step of |g| more."""
from __future__ import annotations

import ctypes

import pytest
import torch

import masked_depthwise_causal_amd as mdc
from masked_depthwise_causal_amd import ssm

from . import ssm_ref as ref
from .gpu_util import announce
from .test_conv_act import DT, dirty, rand
from .test_linear import slack
from .test_ssm_abi import ADDR, INVALID, OK, run, size

F = ref.F
BEND = {"silu": 0.5, "gelu": 1.2, "softplus": 0.25}  # bounds of |act''|


def exact_and_bounds(x, w, b, go, act, pre_type):
    """name: (value, bound) for gx, gw and gbias."""
    dt = x.dtype
    half, half_pre = torch.finfo(dt).eps / 2, torch.finfo(pre_type).eps / 2
    (M, K), N = x.shape, w.shape[0]
    x, w, b, go = (t.to(F) for t in (x, w, b, go))
    pre = x @ w.t() + b
    dp = slack(K) * (x.abs() @ w.abs().t() + b.abs())
    dp = dp + half_pre * (pre.abs() + dp) + torch.finfo(pre_type).tiny
    slope = ref.act_slope(pre, act)
    if act == "relu":
        ds = (pre.abs() <= dp).to(F)
    else:
        ds = BEND[act] * dp + 2.0 ** -21 * (1 + pre.abs())
    g, dg = go * slope, go.abs() * ds
    dr = dg + half * (g.abs() + dg) + torch.finfo(dt).tiny  # with g rounded
    ga = g.abs() + dr
    return {"gx": (g @ w, dr @ w.abs() + slack(N) * (ga @ w.abs())),
            "gw": (g.t() @ x, dr.t() @ x.abs() + slack(M) * (ga.t() @ x.abs())),
            "gbias": (g.sum(0), dg.sum(0) + slack(M) * ga.sum(0))}


def inputs(M, K, N, dtype):
    g = torch.Generator().manual_seed(M + K + N)
    dt = DT[dtype]
    return (rand(g, M, K, dt=dt), rand(g, N, K, dt=dt, scale=K ** -0.5), rand(g, N, dt=dt),
            rand(g, M, N, dt=dt), rand(g, M, N, dt=dt))


SIZES = [(5, 64, 40, "bf16"), (64, 129, 17, "fp16"), (130, 72, 88, "bf16"), (300, 95, 263, "fp16"),
         (130, 1100, 70, "bf16"), (1000, 64, 520, "fp16")]


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N,dtype", SIZES)
@pytest.mark.parametrize("act", ["silu", "gelu", "softplus", "relu"])
def test_gradients_against_the_unrounded_chain(M, K, N, dtype, act):
    x, w, b, res, go = inputs(M, K, N, dtype)
    dev = [t.cuda() for t in (x, w, b)]
    outs = []
    for pre_type in (x.dtype, torch.float32):
        announce(f"linear pre M={M} K={K} N={N} {dtype} {act} pre {pre_type}")
        dirty()
        out, pre = mdc.linear_forward(*dev, activation=act, residual=res.cuda(), return_pre=True,
                                      pre_dtype=pre_type)
        assert pre.dtype == pre_type and pre.shape == (M, N)
        gr = mdc.linear_backward(go.cuda(), *dev[:2], pre, activation=act)
        torch.cuda.synchronize()
        want = exact_and_bounds(x, w, b, go, act, pre_type)
        for got, k in ((gr.x, "gx"), (gr.weight, "gw"), (gr.bias, "gbias")):
            ref.close(got, want[k], 1.0, f"{k}, pre {pre_type}")
        outs.append(out)
        x64, w64 = x.to(F), w.to(F)
        ref.close(pre, (x64 @ w64.t() + b.to(F), x64.abs() @ w64.abs().t() + b.to(F).abs()),
                  slack(K) + 2.0 ** -24, "pre")
    assert torch.equal(*outs)


@pytest.mark.gpu
def test_pre_types_that_are_refused():
    x, w = (torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((6, 32), (24, 32)))
    with pytest.raises(ValueError, match="pre_dtype"):
        mdc.linear_forward(x, w, return_pre=True, pre_dtype=torch.float16)
    with pytest.raises(ValueError, match="pre has dtype"):
        mdc.linear_backward(x[:, :24].contiguous(), x, w, torch.zeros((6, 24), device="cuda").half(),
                            activation="silu")


def args(**kw):
    return ssm.LinearArgs(100, 64, 48, 0, 2, ADDR[0], ADDR[1], ADDR[2], 64, 64, **kw)


def test_abi_checks_an_fp32_pre():
    n = size("mccb_linear_backward_get_workspace_size", args(pre_fp32=1))
    assert n == size("mccb_linear_backward_get_workspace_size", args()) and n[0] == OK
    a = args(pre_fp32=1)
    # two bytes off a float's alignment, and an output inside the second half of its bytes
    assert run("mccb_linear_forward", a, None, 0, ADDR[4], ADDR[5] + 2, ADDR[6], 1 << 30, None) == INVALID
    inside = ADDR[5] + 100 * 48 * 2 + 16
    assert run("mccb_linear_forward", a, None, 0, inside, ADDR[5], ADDR[6], 1 << 30, None) == INVALID
    assert run("mccb_linear_backward", a, ADDR[3], 48, ADDR[4] + 2, ADDR[5], ADDR[6], ADDR[7], ADDR[8], n[1],
               None) == INVALID
    assert run("mccb_linear_backward", a, ADDR[3], 48, ADDR[5], inside, ADDR[6], ADDR[7], ADDR[8], n[1],
               None) == INVALID
    assert ctypes.sizeof(ssm.LinearArgs) % 8 == 0
