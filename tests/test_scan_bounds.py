"""The scan against bounds of fp32 arithmetic that are carried through its recurrences (scan_bounds.py):
close enough to see a state, a decay or a sum that is held in fewer bits."""
from __future__ import annotations

import pytest
import torch

import masked_depthwise_causal_amd as mdc

from . import scan_bounds, ssm_ref as ref
from .gpu_util import announce
from .test_conv_act import dirty
from .test_scan import inputs

NAMES = ("x", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias")


def bounds(v, go, gf, lengths, **kw):
    return scan_bounds.scan(*(v[k] for k in NAMES), lengths, v["state"], go, gf, **kw)


@pytest.mark.parametrize("gate", [False, True])
def test_values_are_the_plain_forms(gate):
    v, go, gf = inputs(21, 2, 12, 5, 3, "bf16", seed=2, gate=gate)
    want = ref.scan(*(v[k] for k in NAMES), True, [21, 8], v["state"], go, gf)
    for k, (value, bound) in bounds(v, go, gf, [21, 8]).items():
        assert torch.allclose(value, want[k][0], rtol=1e-12, atol=1e-12), k
        assert bool((bound >= 0).all())


@pytest.mark.parametrize("S,chunked", [(48, False), (600, True)])
@pytest.mark.parametrize("held", [torch.bfloat16, torch.float16])
def test_bounds_see_a_state_of_16_bits(S, chunked, held):
    """The mistake is in the oracle: its state is rounded after every row."""
    v, go, gf = inputs(S, 1, 24, 8, 1, "fp16", seed=S)
    want = bounds(v, go, gf, None, chunked=chunked)
    got = bounds(v, go, gf, None, chunked=chunked, held=held)
    for k in ("state", "gA"):
        assert bool(((got[k][0] - want[k][0]).abs() > want[k][1]).any()), k


@pytest.mark.gpu
@pytest.mark.parametrize("S,B,H,N,G,dtype,lengths,chunked,parts", [
    (1, 2, 64, 16, 1, "bf16", None, False, {}),
    (16, 2, 70, 8, 1, "fp16", None, False, {"gate": False}),
    (100, 2, 96, 16, 3, "fp16", [100, 67], True, {}),
    (90, 1, 130, 32, 1, "bf16", None, True, {"state": False}),
    (64, 3, 37, 5, 1, "bf16", [64, 0, 49], True, {"bias": False}),
    (700, 1, 40, 16, 1, "fp16", None, True, {}),
    (1100, 1, 64, 4, 1, "bf16", [1030], True, {"gate": False, "skip": False}),
    (300, 9, 1030, 16, 1, "bf16", [300, 299, 0, 1, 300, 16, 17, 160, 300], False, {}),  # enough channels
])
def test_within_what_fp32_may_be_off(S, B, H, N, G, dtype, lengths, chunked, parts):
    v, go, gf = inputs(S, B, H, N, G, dtype, seed=S + N, **parts)
    want = bounds(v, go, gf, lengths, chunked=chunked)
    d = {k: None if t is None else t.cuda() for k, t in v.items()}
    ins = tuple(d[k] for k in ("x", "dt", "A", "Bm", "Cm"))
    opt = {k: d[k] for k in ("D", "z", "dt_bias", "state")}
    opt["lengths"] = None if lengths is None else torch.tensor(lengths, device="cuda")
    announce(f"scan bounds S={S} B={B} H={H} N={N} {dtype}")
    dirty()
    out, fs, saved = mdc.scan_forward(*ins, **opt, return_state=True, return_saved=True)
    gr = mdc.scan_backward(go.cuda(), *ins, saved, **opt, gradFinalState=None if gf is None else gf.cuda())
    torch.cuda.synchronize()
    for k, got in (("out", out), ("state", fs), ("gx", gr.x), ("gdt", gr.dt), ("gA", gr.A), ("gB", gr.B),
                   ("gC", gr.C), ("gD", gr.D), ("gz", gr.z), ("gbias", gr.dt_bias), ("gs", gr.state)):
        if got is not None:
            ref.close(got, want[k], 1.0, k)
