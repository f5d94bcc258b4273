"""Every form that a product takes, forward: few rows with each number of row blocks and waves, each tile
with operands that go straight to LDS and by way of registers, and split contractions. With residual,
pre-activation and bias, since the epilogue's map of threads differs from tile to tile. Tolerances as in
test_linear.py."""
from __future__ import annotations

import pytest
import torch

import masked_depthwise_causal_amd as mdc

from . import ssm_ref as ref
from .gpu_util import announce
from .test_conv_act import DT, dirty, rand
from .test_linear import check, slack, wide

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K,N,dtype,act,extra", [
    # up to 16 rows, 32 and 64; contractions of up to 511, 4095 and more
    (1, 4096, 40, "bf16", "silu", 0),
    (4, 5121, 100, "fp16", "gelu", 0),
    (16, 4103, 64, "bf16", None, 5),
    (3, 1700, 30, "bf16", "softplus", 0),
    (16, 4000, 50, "fp16", "relu", 3),
    (20, 500, 33, "bf16", "silu", 0),
    (20, 1100, 50, "fp16", None, 0),
    (17, 4100, 33, "bf16", "gelu", 0),
    (32, 8192, 24, "fp16", "silu", 8),
    (33, 300, 17, "bf16", "relu", 0),
    (50, 2047, 70, "fp16", "softplus", 0),
    (64, 8000, 48, "bf16", "silu", 0),
])
def test_few_rows(M, K, N, dtype, act, extra):
    check(M, K, N, dtype, act, True, True, extra)


@pytest.mark.parametrize("M,K,N,dtype,act,extra", [
    (4090, 200, 5112, "bf16", "silu", 0),     # 256x320
    (4090, 199, 5101, "fp16", "gelu", 0),     # by way of registers
    (2040, 200, 6136, "fp16", None, 8),       # 256x192
    (2040, 199, 6131, "bf16", "relu", 0),
    (4001, 600, 2040, "bf16", "softplus", 0),  # 128x128
    (4001, 599, 2041, "fp16", "silu", 0),
    (3500, 264, 3700, "fp16", "relu", 8),     # 256x256
    (3500, 263, 3699, "bf16", None, 3),
    (300, 9000, 260, "bf16", "silu", 0),      # 64x64, the contraction over 16 blocks
    (300, 8999, 259, "fp16", "gelu", 0),
    (1024, 4096, 1024, "fp16", "silu", 0),    # 64x64, whole contractions
    (1000, 8192, 2041, "bf16", "silu", 0),
])
def test_tiles(M, K, N, dtype, act, extra):
    g = torch.Generator().manual_seed(M + K + N)
    dt = DT[dtype]
    x, w = rand(g, M, K, dt=dt), rand(g, N, K, dt=dt, scale=K ** -0.5)
    b, res = rand(g, N, dt=dt), rand(g, M, N, dt=dt)
    x64, w64 = x.to(ref.F), w.to(ref.F)
    pre = x64 @ w64.t() + b.to(ref.F)
    mag = x64.abs() @ w64.abs().t() + b.to(ref.F).abs()
    announce(f"linear tiles M={M} K={K} N={N} {dtype} {act} extra={extra}")
    dirty()
    got, gpre = mdc.linear_forward(wide(x, extra, extra // 2), wide(w, extra, extra // 2), b.cuda(), activation=act,
                                   residual=wide(res, extra, 1), return_pre=True)
    torch.cuda.synchronize()
    ref.close(gpre, (pre, mag), slack(K), "pre")
    ref.close(got, (ref.act(pre, act) + res.to(ref.F), mag + res.to(ref.F).abs()), slack(K), "out")
