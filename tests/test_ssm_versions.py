"""Tensors that a call writes in place count it, so that autograd refuses a backward that had saved them."""
from __future__ import annotations

import pytest
import torch

import masked_depthwise_causal_amd as mdc

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def t(*shape, dt=BF):
    return torch.zeros(shape, dtype=dt, device="cuda")


def cases():
    """name: (call, what it writes, what it reads) of every operator that writes a tensor of the caller's."""
    f = torch.float32
    x, w, A, B, q = t(4, 2, 16), t(4, 16), t(8, 16, dt=f), t(4, 2, 8), t(24, 16)
    y, fs, rows, yt = t(4, 2, 16), t(3, 2, 16), t(3, 2, 16), t(2, 16)
    o, st, s, ot, p = t(4, 2, 16), t(2, 8, 16, dt=f), t(2, 8, 16, dt=f), t(2, 16), t(4, 2, 24)
    return {
        "conv forward": (lambda: mdc.conv_act_forward(x, w, y=y, final_state=fs), (y, fs), (x, w)),
        "conv step": (lambda: mdc.conv_act_step(x[0], w, rows, y=yt), (rows, yt), (x, w)),
        "scan forward": (lambda: mdc.scan_forward(x, x, A, B, B, out=o, final_state=st), (o, st), (x, A, B)),
        "scan step": (lambda: mdc.scan_step(s, x[0], x[0], A, B[0], B[0], out=ot), (s, ot), (x, A, B)),
        "linear forward": (lambda: mdc.linear_forward(x, q, out=p), (p,), (x, q)),
    }


@pytest.mark.parametrize("name", ["conv forward", "conv step", "scan forward", "scan step", "linear forward"])
def test_writes_are_counted(name):
    call, written, read = cases()[name]
    before = [v._version for v in written], [v._version for v in read]
    call()
    assert [v._version for v in written] == [n + 1 for n in before[0]]
    assert [v._version for v in read] == before[1]


def test_autograd_sees_that_a_state_moved_on():
    s, x = t(2, 8, 16, dt=torch.float32), t(2, 16)
    leaf = torch.ones_like(s, requires_grad=True)
    loss = (leaf * s).sum()  # saves the state
    mdc.scan_step(s, x, x, t(8, 16, dt=torch.float32), t(2, 8), t(2, 8))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_inference_tensors_are_written_too():
    with torch.inference_mode():
        rows, x, w = t(3, 2, 16), torch.ones((2, 16), dtype=BF, device="cuda"), t(4, 16)
        mdc.conv_act_step(x, w, rows)
        assert bool((rows[-1] == 1).all())
