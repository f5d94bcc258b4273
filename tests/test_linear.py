"""Matrix product with its epilogue against the 64-bit form.

Tolerances. Products of 16-bit values are exact in fp32 and K of them are added in fp32: under
K 2^-24 of mag = sum |x w| + |bias|, whatever the order; the epilogue adds a few roundings and an
activation with a slope below 1.2: (K + 64) 2^-23 mag. The backward takes pre as given; g is
gout act'(pre) with a few fp32 roundings and one to 16 bits (half a step), so sums of its products are
within (half a step + (K + 64) 2^-23) of their magnitudes, K the contraction's length; gbias sums g
before that rounding."""
from __future__ import annotations

import pytest
import torch

import masked_depthwise_causal_amd as mdc

from . import ssm_ref as ref
from .gpu_util import announce
from .test_conv_act import DT, dirty, rand

pytestmark = pytest.mark.gpu
F = ref.F


def slack(K):
    return (K + 64) * 2.0 ** -23


def wide(t, extra, shift):
    """The same values on the device as the middle of wider rows of NaN."""
    if not extra:
        return t.cuda()
    w = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), dtype=t.dtype, device="cuda")
    w[:, shift:shift + t.shape[1]] = t
    return w[:, shift:shift + t.shape[1]]


def check(M, K, N, dtype, act, residual, bias, extra, seed=0):
    g = torch.Generator().manual_seed(seed + M + K + N)
    dt = DT[dtype]
    x, w = rand(g, M, K, dt=dt), rand(g, N, K, dt=dt, scale=K ** -0.5)
    b, res = rand(g, N, dt=dt) if bias else None, rand(g, M, N, dt=dt) if residual else None
    go = rand(g, M, N, dt=dt)
    x64, w64 = x.to(F), w.to(F)
    pre = x64 @ w64.t() + (b.to(F) if bias else 0)
    mag = x64.abs() @ w64.abs().t() + (b.to(F).abs() if bias else 0)
    out = ref.act(pre, act) + (res.to(F) if residual else 0)
    xd, wd, god = wide(x, extra, 1), wide(w, extra, 2), wide(go, extra, 3)
    bd, rd = None if b is None else b.cuda(), None if res is None else wide(res, extra, 1)
    announce(f"linear M={M} K={K} N={N} {dtype} {act} residual={residual} extra={extra}")
    dirty()
    got, gpre = mdc.linear_forward(xd, wd, bd, activation=act, residual=rd, return_pre=True)
    torch.cuda.synchronize()
    ref.close(gpre, (pre, mag), slack(K), "pre")
    ref.close(got, (out, mag + (res.to(F).abs() if residual else 0)), slack(K), "out")
    assert torch.equal(got, mdc.linear_forward(xd, wd, bd, activation=act, residual=rd))
    announce("linear backward")
    grads = mdc.linear_backward(god, xd, wd, gpre, activation=act)
    torch.cuda.synchronize()
    p = gpre.cpu().to(F)
    gg = go.to(F) * ref.act_slope(p, act)
    # slopes are computed in fp32 from terms of up to 1 + |pre|
    gm = go.to(F).abs() * (ref.act_slope(p, act).abs() + 2.0 ** -10 * (1 + p.abs()))
    half = torch.finfo(dt).eps / 2 if act is not None else 0.0
    ref.close(grads.x, (gg @ w64, gm @ w64.abs()), half + slack(N), "gx")
    ref.close(grads.weight, (gg.t() @ x64, gm.t() @ x64.abs()), half + slack(M), "gw")
    ref.close(grads.bias, (gg.sum(0), gm.sum(0)), slack(M), "gbias")
    return xd, wd, bd, rd, god, gpre, got, grads


@pytest.mark.parametrize("M,K,N,dtype,act,residual,bias,extra", [
    (1, 1, 1, "bf16", None, False, False, 0),
    (1, 64, 48, "fp16", "silu", True, True, 0),
    (3, 300, 37, "bf16", "softplus", False, True, 5),
    (16, 129, 16, "fp16", "gelu", True, False, 0),
    (17, 1000, 33, "bf16", "relu", True, True, 3),
    (64, 256, 100, "bf16", None, True, True, 0),
    (65, 7, 9, "fp16", "silu", False, True, 0),          # one tile, padded rows
    (127, 64, 129, "bf16", "gelu", True, True, 8),
    (130, 1100, 70, "fp16", "relu", True, True, 0),      # the contraction split
    (300, 95, 263, "bf16", "softplus", True, True, 5),
    (257, 2056, 128, "bf16", None, False, False, 0),
])
def test_against_64_bits(M, K, N, dtype, act, residual, bias, extra):
    check(M, K, N, dtype, act, residual, bias, extra)


@pytest.mark.parametrize("M,K,N,dtype", [(3500, 200, 3700, "bf16"), (4000, 71, 3601, "fp16")])
def test_large_tiles(M, K, N, dtype):
    """An output large enough for the 256x256 tiles, its last ones partial."""
    check(M, K, N, dtype, "silu", True, True, 0)


@pytest.mark.parametrize("M,K,N,dtype,act", [
    (100, 72, 88, "bf16", "gelu"), (100, 72, 88, "fp16", None),
    (4001, 2040, 600, "bf16", "silu"),   # 128x128 tiles for gx,
    (700, 2040, 4088, "fp16", "relu"),   # for gw
    (3500, 3704, 200, "bf16", "silu"),   # 256x256
    (200, 4088, 4088, "bf16", None),
    (2040, 6136, 72, "fp16", "silu"),    # 256x192
    (200, 6136, 2040, "bf16", "silu"),
    (4090, 5112, 72, "bf16", "relu"),    # 256x320, and gw's contraction split
    (201, 5112, 4088, "fp16", "silu"),
])
def test_backward_reads_operands_as_they_lie(M, K, N, dtype, act):
    """Aligned rows, inside wider ones; every tile, its last ones and the contraction partial."""
    g = torch.Generator().manual_seed(M + K + N)
    dt = DT[dtype]
    x, w, go = rand(g, M, K, dt=dt), rand(g, N, K, dt=dt, scale=K ** -0.5), rand(g, M, N, dt=dt)
    pre = rand(g, M, N, dt=dt)
    announce(f"linear backward M={M} K={K} N={N} {dtype} {act}")
    dirty()
    grads = mdc.linear_backward(wide(go, 16, 8), wide(x, 24, 16), wide(w, 16, 8),
                                None if act is None else pre.cuda(), activation=act)
    torch.cuda.synchronize()
    x64, w64, p, go64 = x.to(F), w.to(F), pre.to(F), go.to(F)
    gg = go64 * ref.act_slope(p, act)
    gm = go64.abs() * (ref.act_slope(p, act).abs() + 2.0 ** -10 * (1 + p.abs()))
    half = torch.finfo(dt).eps / 2 if act is not None else 0.0
    ref.close(grads.x, (gg @ w64, gm @ w64.abs()), half + slack(N), "gx")
    ref.close(grads.weight, (gg.t() @ x64, gm.t() @ x64.abs()), half + slack(M), "gw")
    ref.close(grads.bias, (gg.sum(0), gm.sum(0)), slack(M), "gbias")


def test_leading_dimensions_and_no_rows():
    g = torch.Generator().manual_seed(2)
    x, w, r = rand(g, 5, 3, 32).cuda(), rand(g, 24, 32).cuda(), rand(g, 5, 3, 24).cuda()
    a = mdc.linear_forward(x, w, residual=r)
    b = mdc.linear_forward(x.view(15, 32), w, residual=r.view(15, 24))
    assert a.shape == (5, 3, 24) and torch.equal(a.view(15, 24), b)
    e = torch.empty((0, 32), dtype=torch.bfloat16, device="cuda")
    assert mdc.linear_forward(e, w).shape == (0, 24)
    gr = mdc.linear_backward(torch.empty((0, 24), dtype=torch.bfloat16, device="cuda"), e, w)
    assert gr.x.shape == (0, 32) and not gr.weight.any() and not gr.bias.any()


def test_parts_of_the_gradient():
    xd, wd, _, _, god, pre, _, grads = check(200, 136, 72, "bf16", "silu", False, True, 0, seed=1)
    one = mdc.linear_backward(god, xd, wd, pre, activation="silu", grad_x=False, grad_bias=False)
    assert one.x is None and one.bias is None and torch.equal(one.weight, grads.weight)
    two = mdc.linear_backward(god, xd, wd, pre, activation="silu", grad_weight=False)
    assert two.weight is None and torch.equal(two.x, grads.x) and torch.equal(two.bias, grads.bias)


def test_same_bits_again():
    xd, wd, bd, rd, god, pre, out, grads = check(260, 1500, 140, "fp16", "gelu", True, True, 3, seed=4)
    dirty()
    assert torch.equal(out, mdc.linear_forward(xd, wd, bd, activation="gelu", residual=rd))
    again = mdc.linear_backward(god, xd, wd, pre, activation="gelu")
    assert all(torch.equal(p, q) for p, q in zip(grads, again))
