"""The compiled front end on device tensors: what it refuses before anything is enqueued, what it
accepts, and that a call leaves nothing behind."""
from __future__ import annotations

import gc
import sys

import pytest
import torch

import masked_depthwise_causal_amd as mdc

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def t(*shape, dt=BF):
    return torch.zeros(shape, dtype=dt, device="cuda")


def conv(**kw):
    a = dict(x=t(4, 2, 16), weight=t(4, 16), bias=t(16))
    a.update(kw)
    return mdc.conv_act_forward(**a)


def scan(**kw):
    f = torch.float32
    a = dict(x=t(4, 2, 16), dt=t(4, 2, 16), A=t(8, 16, dt=f), B=t(4, 2, 8), C=t(4, 2, 8), D=t(16, dt=f))
    a.update(kw)
    return mdc.scan_forward(**a)


def linear(**kw):
    a = dict(x=t(6, 32), weight=t(24, 32), bias=t(24))
    a.update(kw)
    return mdc.linear_forward(**a)


@pytest.mark.parametrize("call,kw,error,text", [
    (conv, lambda: dict(weight=t(4, 15)), ValueError, r"weight has shape \(4, 15\), expected \(4, 16\)"),
    (conv, lambda: dict(weight=t(4, 16, dt=torch.float16)), ValueError, "weight has dtype"),
    (conv, lambda: dict(weight=t(16, 4).t()), ValueError, "weight must be contiguous"),
    (conv, lambda: dict(weight=t(5, 16)), mdc.MccbError, None),
    (conv, lambda: dict(x=t(4, 2, 16, dt=torch.float32)), ValueError, "not supported"),
    (conv, lambda: dict(x=t(8, 16)), ValueError, r"\[S,B,H\]"),
    (conv, lambda: dict(lengths=t(2, dt=torch.int32)), ValueError, "lengths has dtype"),
    (conv, lambda: dict(lengths=torch.zeros(2, dtype=torch.int64)), ValueError, "lengths must live on"),
    (conv, lambda: dict(state=t(4, 2, 16)), ValueError, "state has shape"),
    (conv, lambda: dict(y=t(4, 2, 17)), ValueError, "y has shape"),
    (conv, lambda: dict(bias=3.0), TypeError, "bias must be a torch.Tensor"),
    (conv, lambda: dict(activation="gelu"), ValueError, "gelu"),
    (scan, lambda: dict(A=t(8, 16)), ValueError, "A has dtype"),
    (scan, lambda: dict(A=t(33, 16, dt=torch.float32), B=t(4, 2, 33), C=t(4, 2, 33)), mdc.MccbError, None),
    (scan, lambda: dict(B=t(4, 8)), ValueError, "B and C must be"),
    (scan, lambda: dict(C=t(4, 2, 1, 8)), ValueError, "C has shape"),
    (scan, lambda: dict(B=t(4, 2, 3, 8), C=t(4, 2, 3, 8)), mdc.MccbError, None),  # 16 channels in 3 groups
    (scan, lambda: dict(D=t(16)), ValueError, "D has dtype"),
    (scan, lambda: dict(state=t(2, 8, 16)), ValueError, "state has dtype"),
    (linear, lambda: dict(weight=t(24, 31)), ValueError, "weight has shape"),
    (linear, lambda: dict(x=t(6, 64)[:, ::2]), ValueError, "last dimension must be contiguous"),
    (linear, lambda: dict(residual=t(6, 23)), ValueError, "residual has shape"),
    (linear, lambda: dict(x=t(32)), ValueError, "two dimensions"),
])
def test_refuses(call, kw, error, text):
    kw = kw()
    with pytest.raises(error, match=text):
        call(**kw)


def test_refuses_outputs_over_inputs_and_missing_parts():
    x, w = t(4, 2, 16), t(4, 16)
    with pytest.raises(mdc.MccbError):
        mdc.conv_act_forward(x, w, y=x)
    with pytest.raises(mdc.MccbError):
        mdc.linear_backward(t(6, 24), t(6, 32), t(24, 32), None, activation="silu")
    with pytest.raises(ValueError, match="saved has shape"):
        f = torch.float32
        mdc.scan_backward(t(4, 2, 16), t(4, 2, 16), t(4, 2, 16), t(8, 16, dt=f), t(4, 2, 8), t(4, 2, 8),
                          t(3, dt=f))


def test_leaves_nothing_behind():
    """Outputs, workspaces and references, on the good path and on a refusal."""
    x, w = t(6, 32), t(24, 32)
    bad = t(24, 31)

    def once():
        mdc.linear_backward(t(6, 24), x, w, t(6, 24), activation="silu")
        conv(return_state=True)
        scan(return_state=True, return_saved=True)
        with pytest.raises(ValueError):
            linear(weight=bad)

    once()
    gc.collect()
    torch.cuda.synchronize()
    before, counts = torch.cuda.memory_allocated(), [sys.getrefcount(o) for o in (x, w, bad, None)][:3]
    for _ in range(20):
        once()
    gc.collect()
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() == before
    assert [sys.getrefcount(o) for o in (x, w, bad)] == counts
