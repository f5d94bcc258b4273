"""The norms before and after a block against the 64-bit form.

Tolerances relative to the sums of absolute terms (mag). A mean of D squares in fp32, a lane 16 of them and then a tree, is
within 32 2^-24 of itself, its root within half that and the root's own 2^-22; what is made of it passes under ten
roundings of 2^-24 and a sigmoid of 2^-21: 2^-19 for a value, and for a gradient, whose mean is another such sum, 2^-18.
Sums over rows add up to 2^-24 for each row that a block adds in fp32 (8 and up): 2^-18 covers 32, and 2^-17 the largest
here."""
from __future__ import annotations

import pytest
import torch

import masked_depthwise_causal_amd as mdc

from . import delta_ref as ref
from .gpu_util import announce
from .ssm_ref import close
from .test_conv_act import DT, dirty

pytestmark = pytest.mark.gpu


def rand(g, *shape, dt, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).to(dt)


def lay(t, extra):
    """On the device, as a part of rows `extra` wider."""
    wide = torch.cat([t, torch.full((*t.shape[:-1], extra), float("nan"), dtype=t.dtype)], -1).cuda()
    return wide[..., :t.shape[-1]]


SIZES = [(1, 1), (3, 7), (5, 8), (2, 129), (9, 256), (33, 257), (17, 1000), (4, 1024), (70, 1032), (3, 4100), (2, 16384),
         (1500, 64), (2600, 40)]


@pytest.mark.parametrize("R,H", SIZES)
@pytest.mark.parametrize("dtype,residual,scale,extra", [("bf16", True, True, 0), ("fp16", True, False, 3), ("bf16", False, True, 8),
                                                        ("fp16", False, False, 0)])
def test_prenorm(R, H, dtype, residual, scale, extra):
    g = torch.Generator().manual_seed(R + H)
    dt = DT[dtype]
    x, w, go, gs = rand(g, R, H, dt=dt), rand(g, H, dt=dt), rand(g, R, H, dt=dt), rand(g, R, H, dt=dt)
    res = rand(g, R, H, dt=dt, scale=3.0) if residual else None
    sc = rand(g, H, dt=dt) if scale else None
    r = ref.prenorm(x, w, res, sc, gout=go, gsum=gs)
    d = lambda t: None if t is None else lay(t, extra)  # noqa: E731
    announce(f"prenorm R={R} H={H} {dtype}")
    dirty()
    args = {"residual": d(res), "scale": None if sc is None else sc.cuda()}
    xd = d(x)
    out, total = mdc.prenorm_forward(xd, w.cuda(), **args, return_sum=True)
    assert torch.equal(out, mdc.prenorm_forward(xd, w.cuda(), **args))
    close(out, r["out"], 2.0 ** -19, "out")
    close(total, r["sum"], 2.0 ** -22, "sum")
    if not residual and not scale:
        assert total is xd
    gr = mdc.prenorm_backward(d(go), xd, w.cuda(), **args, gradSum=d(gs))
    torch.cuda.synchronize()
    close(gr.x, r["gx"], 2.0 ** -18, "gx")
    close(gr.weight, r["gw"], 2.0 ** -17, "gw")
    assert (gr.residual is None) == (not residual) and (gr.scale is None) == (not scale)
    if residual:
        close(gr.residual, r["gresidual"], 2.0 ** -18, "gresidual")
    if scale:
        close(gr.scale, r["gscale"], 2.0 ** -17, "gscale")
    bare = mdc.prenorm_backward(d(go), xd, w.cuda(), **args)
    close(bare.x, ref.prenorm(x, w, res, sc, gout=go)["gx"], 2.0 ** -18, "gx without gradSum")


@pytest.mark.parametrize("R,H,groups,shared", [(1, 4, 4, True), (5, 48, 3, False), (9, 128, 8, True), (7, 1000, 8, False),
                                               (3, 96, 1, False), (40, 2048, 16, True), (6, 2056, 2, True), (2, 32768, 2, False),
                                               (300, 128, 1, False), (20, 4096, 128, False), (3, 70, 70, True)])
@pytest.mark.parametrize("dtype,gate,residual,scale,extra", [("bf16", True, True, True, 0), ("fp16", True, False, False, 5),
                                                             ("bf16", False, True, False, 8), ("fp16", False, False, True, 0)])
def test_postnorm(R, H, groups, shared, dtype, gate, residual, scale, extra):
    g = torch.Generator().manual_seed(R + H)
    dt = DT[dtype]
    x, go, w = rand(g, R, H, dt=dt), rand(g, R, H, dt=dt), rand(g, H // groups if shared else H, dt=dt)
    z = rand(g, R, H, dt=dt, scale=2.0) if gate else None
    res = rand(g, R, H, dt=dt) if residual else None
    sc = rand(g, H, dt=dt) if scale else None
    r = ref.postnorm(x, w, z, res, sc, groups, gout=go)
    d = lambda t: None if t is None else lay(t, extra)  # noqa: E731
    announce(f"postnorm R={R} H={H} groups={groups} {dtype}")
    dirty()
    args = {"z": d(z), "scale": None if sc is None else sc.cuda(), "groups": groups}
    out = mdc.postnorm_forward(d(x), w.cuda(), residual=d(res), **args)
    close(out, r["out"], 2.0 ** -19, "out")
    gr = mdc.postnorm_backward(d(go), d(x), w.cuda(), **args)
    torch.cuda.synchronize()
    close(gr.x, r["gx"], 2.0 ** -18, "gx")
    close(gr.weight, r["gw"], 2.0 ** -17, "gw")
    assert (gr.z is None) == (not gate) and (gr.scale is None) == (not scale)
    if gate:
        close(gr.z, r["gz"], 2.0 ** -18, "gz")
    if scale:
        close(gr.scale, r["gscale"], 2.0 ** -17, "gscale")


def test_more_axes_and_no_rows():
    w = torch.ones(32, dtype=torch.float16, device="cuda")
    x = torch.randn((3, 4, 32), device="cuda").half()
    a, b = mdc.prenorm_forward(x, w, residual=x), mdc.prenorm_forward(x.view(12, 32), w, residual=x.view(12, 32))
    assert a.shape == x.shape and torch.equal(a.view(12, 32), b)
    time_first = x.transpose(0, 1)[:, 1:2]  # one sequence of a batch: evenly spaced rows
    assert torch.equal(mdc.postnorm_forward(time_first, w), mdc.postnorm_forward(time_first.contiguous(), w))
    e = torch.empty((0, 32), dtype=torch.float16, device="cuda")
    out, total = mdc.prenorm_forward(e, w, residual=e, return_sum=True)
    g = mdc.prenorm_backward(e, e, w, residual=e, scale=w)
    assert out.shape == total.shape == g.x.shape == (0, 32) and not g.weight.any() and not g.scale.any()
    g = mdc.postnorm_backward(e, e, w[:8], z=e, groups=4)
    assert not g.weight.any() and g.weight.shape == (8,)


def test_zero_rows_and_large_values():
    """A row of zeros is normalized with eps alone; rows up to fp32's root of the largest square keep their norm."""
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    x[1] = 1e15
    x[2, 3] = 1e-20
    x[3, :] = torch.arange(64)
    w = torch.full((64,), 2.0, dtype=torch.bfloat16)
    r = ref.postnorm(x, w, gout=torch.ones_like(x))
    out = mdc.postnorm_forward(x.cuda(), w.cuda())
    g = mdc.postnorm_backward(torch.ones_like(x).cuda(), x.cuda(), w.cuda())
    close(out, r["out"], 2.0 ** -19, "out")
    close(g.x, r["gx"], 2.0 ** -18, "gx")
    close(g.weight, r["gw"], 2.0 ** -17, "gw")


def test_outputs_given_and_same_bits():
    g = torch.Generator().manual_seed(1)
    x, z = rand(g, 500, 640, dt=torch.bfloat16).cuda(), rand(g, 500, 640, dt=torch.bfloat16).cuda()
    w = rand(g, 640, dt=torch.bfloat16).cuda()
    y, s = torch.empty_like(x), torch.empty_like(x)
    out, total = mdc.prenorm_forward(x, w, residual=z, return_sum=True, out=y, sum_out=s)
    assert out is y and total is s
    mdc.prenorm_forward(x, w, sum_out=s)
    assert torch.equal(s, x)
    a = mdc.postnorm_backward(z, x, w, z=z, scale=w)
    dirty()
    assert all(torch.equal(p, q) for p, q in zip(a, mdc.postnorm_backward(z, x, w, z=z, scale=w)))


def test_tensors_of_more_than_2_31_values():
    """The last rows, against a call for them alone."""
    R, H, tail = 530_000, 4100, 2000
    x = torch.randn((R, H), device="cuda", dtype=torch.bfloat16)
    z, w = torch.randn((R, H), device="cuda", dtype=torch.bfloat16), torch.randn(H, device="cuda").bfloat16()
    assert x.numel() > 1 << 31
    last = lambda t: t[R - tail:].clone()  # noqa: E731
    announce("norms, more than 2^31 values")
    out, total = mdc.prenorm_forward(x, w, residual=z, return_sum=True)
    out2, total2 = mdc.prenorm_forward(last(x), w, residual=last(z), return_sum=True)
    assert torch.equal(out[R - tail:], out2) and torch.equal(total[R - tail:], total2)
    del out, total
    g = mdc.prenorm_backward(z, x, w)
    assert torch.equal(g.x[R - tail:], mdc.prenorm_backward(last(z), last(x), w).x)
    out = mdc.postnorm_forward(x, w, z=z, groups=4)
    assert torch.equal(out[R - tail:], mdc.postnorm_forward(last(x), w, z=last(z), groups=4))
    del g
    g = mdc.postnorm_backward(out, x, w, z=z, groups=4)
    g2 = mdc.postnorm_backward(last(out), last(x), w, z=last(z), groups=4)
    assert torch.equal(g.x[R - tail:], g2.x) and torch.equal(g.z[R - tail:], g2.z)
