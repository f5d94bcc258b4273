"""Sums of the scan's gradients over many channels and rows."""
from __future__ import annotations

import pytest
import torch

import masked_depthwise_causal_amd as mdc

from .gpu_util import announce
from .test_scan import check

pytestmark = pytest.mark.gpu


def test_sums_over_blocks_of_channels_keep_small_terms():
    """gB and gC of one row are sums of x over the channels here; 62 blocks' sums of 1 lie between one of
    2^24 and one of -2^24, which fp32 additions in that order would swallow."""
    H, G = 64 * 64, 2
    x = torch.zeros((1, 1, G, H), dtype=torch.bfloat16)
    x[..., 7::64] = 1
    x[..., 7], x[..., H - 57] = 2.0 ** 24, -2.0 ** 24
    x = x.view(1, 1, G * H).cuda()
    one = torch.ones((1, 1, G * H), dtype=torch.bfloat16, device="cuda")
    c = torch.ones((1, 1, G, 1), dtype=torch.bfloat16, device="cuda")
    A = -torch.ones((1, G * H), device="cuda")
    announce("scan sums over blocks")
    _, saved = mdc.scan_forward(x, one, A, c, c, softplus=False, return_saved=True)
    g = mdc.scan_backward(one, x, one, A, c, c, saved, softplus=False)
    assert g.C.flatten().tolist() == [62.0, 62.0] and g.B.flatten().tolist() == [62.0, 62.0]


@pytest.mark.parametrize("S,B,H,N,G,dtype,lengths", [
    (20, 1, 4160, 16, 1, "bf16", None),          # 65 blocks of channels
    (17, 2, 2500, 6, 1, "fp16", [17, 9]),
    (600, 8, 1100, 16, 1, "bf16", [600, 555, 600, 0, 512, 513, 600, 1]),  # not cut: more than 32 tiles
])
def test_many_channels_and_rows(S, B, H, N, G, dtype, lengths):
    check(S, B, H, N, G, dtype, lengths, seed=S)
