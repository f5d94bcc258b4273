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
from .test_delta import inputs, slack

pytestmark = pytest.mark.gpu


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
