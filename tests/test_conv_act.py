"""Causal convolution with activation and carried rows against the 64-bit form.

Tolerances. Products of 16-bit values are exact in fp32. y: W+1 fp32 roundings of terms below
mag = |bias| + sum |w x|, then silu: exp2, reciprocal and products, each within 2^-22, whose slope is
below 1.1: under 16 units of 2^-24 each in all, 2^-20 mag. Gradients: g carries the same 2^-20 of
|gy| (1.1 + mag) (its slope's slope is below 1); gx adds W+1 roundings; gw and gbias add fp32 sums
over a strip of at most 128 rows (128 roundings, 2^-17) and fp64 beyond. Each result is then rounded
once to its type."""
from __future__ import annotations

import pytest
import torch

import masked_depthwise_causal_amd as mdc

from . import ssm_ref as ref
from .gpu_util import announce

pytestmark = pytest.mark.gpu

Y, GX, GSUM = 2.0 ** -20, 2.0 ** -19, 2.0 ** -16
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def dirty(n=1 << 22):
    """Leaves NaN in the allocator's free blocks: outputs and workspaces need no initial values."""
    for size in (n, n // 64):
        torch.full((size,), float("nan"), device="cuda")


def rand(g, *shape, dt=torch.bfloat16, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).to(dt)


def lay(t, layout):
    """The same values on the device as a strided view."""
    t = t.cuda()
    if layout == "contig":
        return t
    if layout == "batch_first":  # [B,S,H] storage
        return t.transpose(0, 1).contiguous().transpose(0, 1)
    if layout == "slice":  # the middle of wider rows, off every alignment
        S, B, H = t.shape
        wide = torch.full((S, B, 2 * H + 3), float("nan"), dtype=t.dtype, device="cuda")
        wide[:, :, 1:H + 1] = t
        return wide[:, :, 1:H + 1]
    if layout == "channels_apart":
        wide = torch.full((*t.shape, 2), float("nan"), dtype=t.dtype, device="cuda")
        wide[..., 0] = t
        return wide[..., 0]
    raise ValueError(layout)


def case(S, B, H, W, dtype, kind, lengths, with_state, with_bias, layout, seed):
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    x, gy = rand(g, S, B, H, dt=dt), rand(g, S, B, H, dt=dt)
    w, bias = rand(g, W, H, dt=dt, scale=0.6), rand(g, H, dt=dt) if with_bias else None
    state = rand(g, W - 1, B, H, dt=dt) if with_state else None
    gf = rand(g, W - 1, B, H, dt=dt) if with_state else None
    r = ref.conv(x, w, bias, kind, lengths, state, gy, gf)
    for b, n in enumerate(ref.lens_of(lengths, S, B)):  # what dead rows hold must not matter
        x[n:, b], gy[n:, b] = float("nan"), float("inf")
    dev = {"lengths": None if lengths is None else torch.tensor(lengths, device="cuda"),
           "state": None if state is None else state.cuda(), "activation": kind}
    xd, gyd, wd = lay(x, layout), lay(gy, layout), w.cuda()
    bd = None if bias is None else bias.cuda()
    announce(f"conv_act S={S} B={B} H={H} W={W} {dtype} {kind} {lengths} {layout}")
    dirty()
    y, fs = mdc.conv_act_forward(xd, wd, bd, return_state=True, **dev)
    gr = mdc.conv_act_backward(gyd, xd, wd, bd, gradFinalState=None if gf is None else gf.cuda(), **dev)
    torch.cuda.synchronize()
    ref.close(y, r["y"], Y, "y")
    assert torch.equal(fs.cpu().to(ref.F), r["state"][0]), "final state"
    ref.close(gr.x, r["gx"], GX, "gx")
    ref.close(gr.weight, r["gw"], GSUM, "gw")
    if bias is not None:
        ref.close(gr.bias, r["gb"], GSUM, "gbias")
    if state is not None:
        ref.close(gr.state, r["gs"], GX, "gstate")
    return xd, gyd, wd, bd, dev, y, fs, gr


@pytest.mark.parametrize("S,B,H,W,dtype,kind,lengths,with_state,with_bias,layout", [
    (1, 1, 1, 4, "bf16", "silu", None, True, True, "contig"),
    (2, 3, 7, 4, "fp16", "silu", None, True, True, "contig"),
    (5, 2, 8, 3, "bf16", None, None, False, False, "contig"),
    (37, 3, 65, 2, "fp16", "silu", [0, 1, 37], True, True, "slice"),
    (129, 2, 100, 4, "bf16", "silu", [129, 2], True, True, "batch_first"),
    (64, 2, 24, 4, "bf16", "silu", [63, 0], True, False, "channels_apart"),
    (300, 1, 133, 1, "fp16", "silu", None, True, True, "contig"),
    (131, 4, 512, 4, "fp16", "silu", [131, 128, 127, 3], False, True, "contig"),
    (257, 2, 384, 3, "bf16", None, [200, 1000], True, True, "slice"),  # a length past S counts as S
])
def test_against_64_bits(S, B, H, W, dtype, kind, lengths, with_state, with_bias, layout):
    case(S, B, H, W, dtype, kind, lengths, with_state, with_bias, layout, seed=S + H)


def test_no_rows():
    w, s = torch.ones((3, 16), dtype=torch.bfloat16, device="cuda"), \
        torch.randn((2, 2, 16), device="cuda").bfloat16()
    x = torch.empty((0, 2, 16), dtype=torch.bfloat16, device="cuda")
    y, fs = mdc.conv_act_forward(x, w, state=s, return_state=True)
    assert y.shape == (0, 2, 16) and torch.equal(fs, s)
    gf = torch.randn((2, 2, 16), device="cuda").bfloat16()
    gr = mdc.conv_act_backward(x, x, w, state=s, gradFinalState=gf)
    assert torch.equal(gr.state, gf) and not gr.weight.any()


def test_plain_form_equals_the_framework_forward():
    # without bias and activation this is the convolution of mdc.forward: both round the same sum
    g = torch.Generator().manual_seed(3)
    x, w = rand(g, 70, 2, 384).cuda(), rand(g, 3, 384, scale=0.5).cuda()
    a, b = mdc.conv_act_forward(x, w, activation=None), mdc.forward(x, w)
    d = (a.float() - b.float()).abs()
    assert bool((d <= 2.0 ** -8 * b.float().abs() + 2.0 ** -20).all())


@pytest.mark.parametrize("H,W,dtype", [(7, 4, "bf16"), (64, 3, "fp16"), (133, 2, "bf16"), (16, 1, "fp16")])
def test_tokens_continue_a_prompt(H, W, dtype):
    """A prompt cut in two, then single tokens, equals the whole prompt: bit for bit, since every
    row's sum has one order in all forms."""
    g = torch.Generator().manual_seed(H)
    S, B, dt = 23, 3, DT[dtype]
    x, w, b = rand(g, S, B, H, dt=dt).cuda(), rand(g, W, H, dt=dt).cuda(), rand(g, H, dt=dt).cuda()
    announce(f"conv tokens H={H} W={W}")
    whole, end = mdc.conv_act_forward(x, w, b, return_state=True)
    y0, st = mdc.conv_act_forward(x[:5], w, b, return_state=True)
    y1, st = mdc.conv_act_forward(x[5:17], w, b, state=st, return_state=True)
    parts = [y0, y1] + [mdc.conv_act_step(x[t], w, st, b)[None] for t in range(17, S)]
    assert torch.equal(torch.cat(parts), whole)
    assert torch.equal(st, end)


def test_token_with_strided_row():
    g = torch.Generator().manual_seed(4)
    x = rand(g, 3, 40).cuda()
    w, s = rand(g, 4, 20).cuda(), rand(g, 3, 3, 20).cuda()
    a, b = s.clone(), s.clone()
    y = mdc.conv_act_step(x[:, 1::2], w, a)
    z = mdc.conv_act_step(x[:, 1::2].contiguous(), w, b)
    assert torch.equal(y, z) and torch.equal(a, b)


def test_same_bits_again():
    xd, gyd, wd, bd, dev, y, fs, gr = case(200, 2, 136, 4, "bf16", "silu", [200, 77], True, True,
                                           "slice", seed=5)
    dirty()
    y2, fs2 = mdc.conv_act_forward(xd, wd, bd, return_state=True, **dev)
    g2 = mdc.conv_act_backward(gyd, xd, wd, bd, **dev)
    g3 = mdc.conv_act_backward(gyd, xd, wd, bd, **dev)
    assert torch.equal(y, y2) and torch.equal(fs, fs2)
    assert all(torch.equal(p, q) for p, q in zip(g2, g3))
