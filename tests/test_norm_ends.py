"""The norms at the ends of what they take."""
from __future__ import annotations

import pytest
import torch

import masked_depthwise_causal_amd as mdc

from .test_delta_abi import ADDR, INVALID, norm, run, size


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
