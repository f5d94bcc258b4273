"""The state space block's operators at sizes whose elements, or threads, pass 32 bits: refused before
anything is enqueued, or computed."""
from __future__ import annotations

import pytest
import torch

import masked_depthwise_causal_amd as mdc

from .gpu_util import announce
from .test_ssm_abi import OK, SHAPE, scan, size

BF = torch.bfloat16


@pytest.mark.parametrize("name", ["mccb_scan_saved_size", "mccb_scan_forward_get_workspace_size",
                                  "mccb_scan_backward_get_workspace_size"])
def test_more_groups_than_a_grid_has_blocks(name):
    def rc(G, H, N):
        return size(name, scan(S=1, B=1, H=H, N=N, G=G))[0]

    assert rc(1 << 23, 1 << 23, 32) == SHAPE
    assert rc(1 << 24, 1 << 24, 1) == SHAPE
    assert rc(1 << 22, 1 << 24, 32) == OK


@pytest.mark.gpu
def test_scan_gradients_of_two_to_the_32_coefficients():
    """gB and gC of 2^24 rows in 8 groups of 16 places: two halves of the batch that are alike, and the same
    as half of the batch gives alone."""
    S, B, G, N = 1 << 18, 64, 8, 9
    g = torch.Generator(device="cuda").manual_seed(1)
    one = [torch.randn((S, B // 2, G), generator=g, device="cuda").to(BF) for _ in range(3)]
    x, dt, go = (torch.cat([t, t], 1) for t in one)
    Bm, Cm = (torch.randn((1, 1, G, N), generator=g, device="cuda").to(BF) for _ in range(2))
    A = -torch.rand((N, G), generator=g, device="cuda") - 0.1

    def grads(x, dt, go):
        n = x.shape[1]
        b, c = Bm.expand(S, n, G, N), Cm.expand(S, n, G, N)
        _, saved = mdc.scan_forward(x, dt, A, b, c, return_saved=True)
        r = mdc.scan_backward(go, x, dt, A, b, c, saved)
        torch.cuda.synchronize()
        return r

    announce("scan of half of the batch")
    want = grads(*one)
    announce("scan of the batch")
    got = grads(x, dt, go)
    assert torch.isfinite(want.B).all() and want.B.any() and want.C.any()
    for name in ("B", "C", "x", "dt"):
        a, b = getattr(got, name), getattr(want, name)
        assert torch.equal(a[:, :B // 2], b) and torch.equal(a[:, B // 2:], b), name


@pytest.mark.gpu
def test_conv_gradients_of_many_channels_apart():
    """2^30 channels of one row, each a lane's own since they are not adjacent."""
    B, H = 65535, 16386
    g = torch.Generator(device="cuda").manual_seed(2)
    x, gy = (torch.randn((1, B, 1), generator=g, device="cuda").to(BF) for _ in range(2))
    w = torch.randn((1, H), generator=g, device="cuda").to(BF)
    announce("conv backward of 2^30 channels")
    r = mdc.conv_act_backward(gy.expand(1, B, H), x.expand(1, B, H), w, activation=None)
    torch.cuda.synchronize()
    for b in range(0, B, 4096):  # a product of two 16-bit values is exact in fp32
        assert torch.equal(r.x[0, b:b + 4096], (gy[0, b:b + 4096].float() * w.float()).to(BF))
    # sums of exact products, in fp64 over the batch, rounded once to fp32 and once to 16 bits
    want = float((gy.double() * x.double()).sum())
    assert bool((r.weight.double() - want).abs().max() <= 2.0 ** -8 * (1 + 2.0 ** -10) * abs(want))
    assert bool((r.weight == r.weight[0, 0]).all())


@pytest.mark.gpu
def test_weight_gradient_of_no_rows_and_two_to_the_32_elements():
    n = 65536
    w = torch.ones((1, n), dtype=BF, device="cuda").expand(n, n)
    e = torch.empty((0, n), dtype=BF, device="cuda")
    torch.full((n * n // 2,), float("nan"), device="cuda")  # what the gradient's memory held
    announce("linear backward of no rows")
    r = mdc.linear_backward(e, e, w)
    torch.cuda.synchronize()
    assert r.weight.shape == (n, n) and not r.weight.any() and not r.bias.any()
