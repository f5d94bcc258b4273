"""How the state space block's operators are called: the stream they run on, and flags."""
from __future__ import annotations

import pytest
import torch

import masked_depthwise_causal_amd as mdc

from .gpu_util import announce

BF = torch.bfloat16


def test_refuses_a_stream_of_another_device():
    class Stream:
        device = torch.device("cuda", 1)

    x, w = torch.zeros((4, 2, 8), dtype=BF), torch.zeros((4, 8), dtype=BF)
    with pytest.raises(ValueError, match="stream lives on cuda:1"):
        mdc.conv_act_forward(x, w, stream=Stream())
    with pytest.raises(ValueError, match="stream lives on cuda:1"):
        mdc.linear_forward(x, w, stream=Stream())


def calls(v, stream=None):
    """Every operator on the inputs `v`, none of them on another's result."""
    c = mdc.conv_act_forward(v["x"], v["w"], stream=stream)
    cg = mdc.conv_act_backward(v["go"], v["x"], v["w"], stream=stream)
    ct = mdc.conv_act_step(v["x"][0], v["w"], v["rows"], stream=stream)
    o, saved = mdc.scan_forward(v["x"], v["dt"], v["A"], v["B"], v["C"], return_saved=True, stream=stream)
    og = mdc.scan_backward(v["go"], v["x"], v["dt"], v["A"], v["B"], v["C"], v["saved"], stream=stream)
    ot = mdc.scan_step(v["state"], v["x"][0], v["dt"][0], v["A"], v["B"][0], v["C"][0], stream=stream)
    p = mdc.linear_forward(v["x"], v["q"], activation="silu", stream=stream)
    pg = mdc.linear_backward(v["gq"], v["x"], v["q"], v["pre"], activation="silu", stream=stream)
    return {"conv_act_forward": c, "conv_act_step": ct, "rows": v["rows"], "scan_forward": o, "saved": saved,
            "scan_step": ot, "state": v["state"], "linear_forward": p,
            **{f"conv_act_backward {i}": t for i, t in enumerate(cg) if t is not None},
            **{f"scan_backward {i}": t for i, t in enumerate(og) if t is not None},
            **{f"linear_backward {i}": t for i, t in enumerate(pg)}}


def values(seed):
    g = torch.Generator().manual_seed(seed)
    S, B, H, N, Q = 70, 2, 96, 8, 40

    def r(*shape, dt=BF):
        return torch.randn(shape, generator=g).to(dt).cuda()

    return {"x": r(S, B, H), "dt": r(S, B, H), "go": r(S, B, H), "w": r(4, H), "rows": r(3, B, H),
            "A": -r(N, H, dt=torch.float32).abs() - 0.1, "B": r(S, B, N), "C": r(S, B, N),
            "state": r(B, N, H, dt=torch.float32), "q": r(Q, H), "gq": r(S, B, Q), "pre": r(S, B, Q),
            "saved": r((S + 15) // 16 * B * N * H, dt=torch.float32)}


@pytest.mark.gpu
def test_calls_run_on_the_stream_that_is_given():
    """On the side stream the inputs are rewritten after a delay, so a call that ran anywhere else would
    read what they held before."""
    old, new = values(1), values(2)
    want = {k: t.clone() for k, t in calls({k: t.clone() for k, t in new.items()}).items()}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    announce("calls behind a delay on a side stream")
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)  # about 50 ms; the calls below are enqueued in one
        for k in old:
            old[k].copy_(new[k])
    got = calls(old, side)
    side.synchronize()
    for k in want:
        assert torch.equal(got[k], want[k]), k


def test_flags_are_read_before_anything_runs():
    """A flag without a truth value is refused first, not once the kernels are enqueued."""
    x, c = torch.zeros((4, 2, 8), dtype=BF), torch.zeros((4, 2, 1), dtype=BF)
    A = torch.zeros((1, 8))
    flag = torch.zeros(2)
    with pytest.raises(RuntimeError, match="Boolean value"):
        mdc.scan_forward(x, x, A, c, c, softplus=flag)
    with pytest.raises(RuntimeError, match="Boolean value"):
        mdc.scan_backward(x, x, x, A, c, c, c, softplus=flag)
    with pytest.raises(RuntimeError, match="Boolean value"):
        mdc.scan_step(torch.zeros((2, 1, 8)), x[0], x[0], A, c[0], c[0], softplus=flag)
