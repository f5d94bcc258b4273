"""The norms at the ends of what they take."""
from __future__ import annotations

import pytest
import torch

import masked_depthwise_causal_amd as mdc

from . import delta_ref as ref
from .gpu_util import announce
from .ssm_ref import close
from .test_conv_act import DT
from .test_delta_abi import ADDR, INVALID, norm, run, size
from .test_norms import lay, rand


@pytest.mark.parametrize("eps", [2.0 ** -127, 1e-44])
def test_refuses_an_eps_that_the_root_takes_for_zero(eps):
    a = norm(eps=eps, residual=None, scale=None)
    assert run("mccb_prenorm_forward", a, ADDR[4], ADDR[6], None) == INVALID
    assert run("mccb_postnorm_forward", a, ADDR[4], None) == INVALID
    assert run("mccb_prenorm_backward", a, ADDR[4], 24, None, 24, ADDR[6], None, ADDR[7], None, ADDR[10], 1 << 20, None) == INVALID
    assert run("mccb_postnorm_backward", a, ADDR[4], 24, ADDR[6], None, ADDR[7], None, ADDR[10], 1 << 20, None) == INVALID
    assert size("mccb_prenorm_backward_get_workspace_size", a)[0] == INVALID


@pytest.mark.gpu
def test_rows_of_zeros_with_the_smallest_eps():
    x = torch.zeros((2, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    for eps in (1e-30, 2.0 ** -126):
        assert not mdc.prenorm_forward(x, w, eps=eps).any() and not mdc.postnorm_forward(x, w, eps=eps).any()
        assert torch.isfinite(mdc.prenorm_backward(x + 1, x, w, eps=eps).x).all()
    with pytest.raises(mdc.MccbError):
        mdc.prenorm_forward(x, w, eps=1e-44)


@pytest.mark.gpu
@pytest.mark.parametrize("R,H,groups,dtype,extra", [(300, 8200, 1, "bf16", 0), (130, 16384, 1, "fp16", 8), (61, 18010, 2, "bf16", 3)])
def test_wide_groups(R, H, groups, dtype, extra):
    """Gradients over groups of more than 8192 values, with more rows than one block takes; bounds of test_norms.py, as a
    block adds 4 rows here."""
    g = torch.Generator().manual_seed(R)
    dt = DT[dtype]
    x, go, z, w, sc = rand(g, R, H, dt=dt), rand(g, R, H, dt=dt), rand(g, R, H, dt=dt), rand(g, H, dt=dt), rand(g, H, dt=dt)
    announce(f"wide groups R={R} H={H}")
    r = ref.postnorm(x, w, z, None, sc, groups, gout=go)
    gr = mdc.postnorm_backward(lay(go, extra), lay(x, extra), w.cuda(), z=lay(z, extra), scale=sc.cuda(), groups=groups)
    close(gr.x, r["gx"], 2.0 ** -18, "gx")
    close(gr.z, r["gz"], 2.0 ** -18, "gz")
    close(gr.weight, r["gw"], 2.0 ** -17, "gw")
    close(gr.scale, r["gscale"], 2.0 ** -17, "gscale")
    if groups == 1:
        r = ref.prenorm(x, w, z, sc, gout=go, gsum=x)
        gr = mdc.prenorm_backward(lay(go, extra), lay(x, extra), w.cuda(), residual=lay(z, extra), scale=sc.cuda(), gradSum=lay(x, extra))
        close(gr.x, r["gx"], 2.0 ** -18, "gx")
        close(gr.residual, r["gresidual"], 2.0 ** -18, "gresidual")
        close(gr.weight, r["gw"], 2.0 ** -17, "gw")
        close(gr.scale, r["gscale"], 2.0 ** -17, "gscale")
