"""The state space block's C-ABI without a GPU: exports, workspace sizes, and refusals. Every call that
passes made-up addresses is one that the host-side checks must reject before any HIP call."""
from __future__ import annotations

import ctypes
import os
import re
import subprocess

import pytest
import torch

import masked_depthwise_causal_amd as mdc
from masked_depthwise_causal_amd import build as mbuild
from masked_depthwise_causal_amd import ssm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mccb_ssm.h")
OK, NULLPTR, INVALID, SHAPE = mdc.MCCB_OK, mdc.MCCB_ERR_PARAM_NULLPTR, mdc.MCCB_ERR_PARAM_INVALID, \
    mdc.MCCB_ERR_SHAPE
GB = 1 << 30
ADDR = [0x7E0000000000 + k * 16 * GB for k in range(24)]  # never dereferenced


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(mccb_[a-z_]+)\s*\(", text)))


def test_exports_every_declared_function():
    lib = ssm.ssm_lib()
    assert set(declared()) == set(ssm._SIGNATURES)
    out = subprocess.run(["nm", "-D", "--defined-only", mbuild.SSM_LIB], capture_output=True,
                         text=True, check=True).stdout
    assert set(declared()) <= set(re.findall(r"\bT (mccb_\w+)", out))
    assert all(hasattr(lib, n) for n in declared())


def test_struct_sizes_match_the_header(tmp_path):
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include "mccb_ssm.h"\nint main(void) { printf("%zu %zu %zu %zu",'
                   "sizeof(mccb_conv_t), sizeof(mccb_scan_t), sizeof(mccb_scan_grads_t), "
                   "sizeof(mccb_linear_t)); return 0; }\n")
    exe = str(tmp_path / "sizes")
    subprocess.run(["gcc", "-std=c11", "-I", mbuild.INCLUDE, str(src), "-o", exe], check=True)
    got = [int(v) for v in subprocess.run([exe], capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(t) for t in
                   (ssm.ConvArgs, ssm.ScanArgs, ssm.ScanGradArgs, ssm.LinearArgs)]


def run(name, args, *rest):
    rc = getattr(ssm.ssm_lib(), name)(ctypes.addressof(args) if args is not None else None, *rest)
    assert rc != OK, f"{name} passed its checks with made-up addresses"
    return rc


def size(name, args):
    out = ctypes.c_uint64(0)
    rc = getattr(ssm.ssm_lib(), name)(ctypes.addressof(args), ctypes.addressof(out))
    return rc, out.value


# -- convolution -------------------------------------------------------------------------------------
def conv(S=8, B=2, H=16, W=4, dtype=0, activation=2, x=ADDR[0], strides=(32, 16, 1), weight=ADDR[1],
         bias=ADDR[2], lengths=ADDR[3], state=ADDR[4]):
    return ssm.ConvArgs(S, B, H, W, dtype, activation, x, *strides, weight, bias, lengths, state)


def conv_forward(y=ADDR[5], final=ADDR[6], **kw):
    return run("mccb_conv_act_forward", conv(**kw), y, final, None)


def conv_backward(gy=ADDR[7], gfinal=ADDR[8], gx=ADDR[9], gw=ADDR[10], gb=ADDR[11], gs=ADDR[12],
                  ws=ADDR[13], wsz=None, gstride=(32, 16, 1), **kw):
    a = conv(**kw)
    if wsz is None:
        wsz = size("mccb_conv_act_backward_get_workspace_size", a)[1]
    st = (ctypes.c_int64 * 3)(*gstride)
    return run("mccb_conv_act_backward", a, gy, ctypes.addressof(st), gfinal, gx, gw, gb, gs, ws, wsz,
               None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), NULLPTR), (dict(weight=None), NULLPTR), (dict(y=None), NULLPTR),
    (dict(dtype=2), INVALID), (dict(activation=1), INVALID), (dict(activation=9), INVALID),
    (dict(W=0), SHAPE), (dict(W=5), SHAPE), (dict(B=0), SHAPE), (dict(H=0), SHAPE),
    (dict(S=-1), SHAPE), (dict(S=1 << 31), SHAPE), (dict(B=60000, H=1 << 20), SHAPE),
    (dict(strides=(-32, 16, 1)), INVALID), (dict(strides=(1 << 62, 16, 1)), INVALID),
    (dict(x=ADDR[0] + 1), INVALID), (dict(lengths=ADDR[3] + 4), INVALID), (dict(y=ADDR[5] + 1), INVALID),
    (dict(y=ADDR[0] + 64), INVALID), (dict(y=ADDR[1]), INVALID), (dict(final=ADDR[4]), INVALID),
    (dict(final=ADDR[5] + 16), INVALID)])
def test_conv_forward_refuses(kw, code):
    assert conv_forward(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(gy=None), NULLPTR), (dict(gx=None), NULLPTR), (dict(gw=None), NULLPTR), (dict(ws=None), NULLPTR),
    (dict(wsz=0), INVALID), (dict(ws=ADDR[13] + 8), INVALID), (dict(gx=ADDR[7]), INVALID),
    (dict(gs=ADDR[8]), INVALID), (dict(gb=ADDR[10]), INVALID), (dict(ws=ADDR[9]), INVALID),
    (dict(gstride=(32, -1, 1)), INVALID), (dict(activation=3), INVALID)])
def test_conv_backward_refuses(kw, code):
    assert conv_backward(**kw) == code


@pytest.mark.parametrize("kw,state,y,code", [
    (dict(), None, ADDR[5], NULLPTR), (dict(), ADDR[4], None, NULLPTR), (dict(S=2), ADDR[4], ADDR[5], SHAPE),
    (dict(lengths=ADDR[3]), ADDR[4], ADDR[5], INVALID), (dict(state=ADDR[6]), ADDR[4], ADDR[5], INVALID),
    (dict(), ADDR[4], ADDR[4], INVALID), (dict(), ADDR[0], ADDR[5], INVALID)])
def test_conv_step_refuses(kw, state, y, code):
    a = conv(**{"S": 1, "lengths": None, "state": None, **kw})
    assert run("mccb_conv_act_step", a, state, y, None) == code


# -- scan --------------------------------------------------------------------------------------------
def scan(S=8, B=2, H=16, N=4, G=2, dtype=0, softplus=1, x=ADDR[0], dt=ADDR[1], z=ADDR[2], Bm=ADDR[3],
         Cm=ADDR[4], rows=(32, 16, 1), coef=(16, 8, 4, 1), A=ADDR[5], D=ADDR[6], bias=ADDR[7],
         lengths=ADDR[8], state=ADDR[9]):
    return ssm.ScanArgs(S, B, H, N, G, dtype, softplus, x, dt, z, Bm, Cm, *rows, *rows, *rows, *coef,
                        *coef, A, D, bias, lengths, state)


def scan_forward(out=ADDR[10], final=ADDR[11], saved=ADDR[12], ws=ADDR[13], wsz=1 << 30, **kw):
    return run("mccb_scan_forward", scan(**kw), out, final, saved, ws, wsz, None)


GRADS = dict(go=ADDR[10], gfinal=ADDR[11], gx=ADDR[12], gdt=ADDR[13], gz=ADDR[14], gB=ADDR[15],
             gC=ADDR[16], gA=ADDR[17], gD=ADDR[18], gb=ADDR[19], gs=ADDR[20])


def scan_backward(saved=ADDR[21], ws=ADDR[22], wsz=None, **kw):
    g = {k: kw.pop(k, v) for k, v in GRADS.items()}
    a = scan(**kw)
    if wsz is None:
        wsz = size("mccb_scan_backward_get_workspace_size", a)[1]
    grads = ssm.ScanGradArgs(g["go"], 32, 16, 1, *list(g.values())[1:])
    return run("mccb_scan_backward", a, ctypes.addressof(grads), saved, ws, wsz, None)


@pytest.mark.parametrize("kw,code", [
    *((dict([(k, None)]), NULLPTR) for k in ("x", "dt", "Bm", "Cm", "A", "out")),
    (dict(dtype=-1), INVALID), (dict(N=0), SHAPE), (dict(N=33), SHAPE), (dict(G=0), SHAPE),
    (dict(G=3), SHAPE), (dict(B=70000), SHAPE), (dict(S=-3), SHAPE), (dict(rows=(32, 16, -1)), INVALID),
    (dict(coef=(16, 8, -4, 1)), INVALID), (dict(A=ADDR[5] + 2), INVALID), (dict(state=ADDR[9] + 2), INVALID),
    (dict(z=ADDR[2] + 1), INVALID), (dict(saved=ADDR[12] + 4), INVALID), (dict(out=ADDR[2]), INVALID),
    (dict(final=ADDR[9]), INVALID), (dict(out=ADDR[12]), INVALID), (dict(final=ADDR[5] + 128), INVALID)])
def test_scan_forward_refuses(kw, code):
    assert scan_forward(**kw) == code


def test_scan_forward_needs_its_workspace():
    a = dict(S=4096, B=1, H=64, G=1, rows=(64, 64, 1), coef=(4, 4, 4, 1))
    rc, need = size("mccb_scan_forward_get_workspace_size", scan(**a))
    assert rc == OK and need > 0  # a long sequence of few channels is cut into chunks
    assert scan_forward(ws=None, wsz=need, **a) == NULLPTR
    assert scan_forward(wsz=need - 1, **a) == INVALID
    assert scan_forward(ws=ADDR[0], wsz=need, **a) == INVALID


@pytest.mark.parametrize("kw,code", [
    *((dict([(k, None)]), NULLPTR) for k in ("go", "gx", "gdt", "gz", "gB", "gC", "gA", "saved", "ws")),
    (dict(z=None), INVALID), (dict(gA=ADDR[17] + 2), INVALID), (dict(gx=ADDR[13]), INVALID),
    (dict(gB=ADDR[3]), INVALID), (dict(gs=ADDR[9]), INVALID), (dict(gx=ADDR[10]), INVALID),
    (dict(wsz=16), INVALID), (dict(ws=ADDR[21]), INVALID), (dict(saved=ADDR[21] + 8), INVALID)])
def test_scan_backward_refuses(kw, code):
    assert scan_backward(**kw) == code


@pytest.mark.parametrize("kw,state,out,code", [
    (dict(), None, ADDR[10], NULLPTR), (dict(), ADDR[9], None, NULLPTR), (dict(S=2), ADDR[9], ADDR[10], SHAPE),
    (dict(state=ADDR[11]), ADDR[9], ADDR[10], INVALID), (dict(lengths=ADDR[8]), ADDR[9], ADDR[10], INVALID),
    (dict(), ADDR[9] + 2, ADDR[10], INVALID), (dict(), ADDR[9], ADDR[9] + 64, INVALID),
    (dict(), ADDR[9], ADDR[0], INVALID)])
def test_scan_step_refuses(kw, state, out, code):
    a = scan(**{"S": 1, "lengths": None, "state": None, **kw})
    assert run("mccb_scan_step", a, state, out, None) == code


# -- matrix product ----------------------------------------------------------------------------------
def linear(M=100, K=64, N=48, dtype=0, activation=2, x=ADDR[0], weight=ADDR[1], bias=ADDR[2], x_ld=64,
           w_ld=64):
    return ssm.LinearArgs(M, K, N, dtype, activation, x, weight, bias, x_ld, w_ld)


def linear_forward(res=ADDR[3], res_ld=48, out=ADDR[4], pre=ADDR[5], ws=ADDR[6], wsz=1 << 30, **kw):
    return run("mccb_linear_forward", linear(**kw), res, res_ld, out, pre, ws, wsz, None)


def linear_backward(go=ADDR[3], go_ld=48, pre=ADDR[4], gx=ADDR[5], gw=ADDR[6], gb=ADDR[7], ws=ADDR[8],
                    wsz=None, **kw):
    a = linear(**kw)
    if wsz is None:
        wsz = size("mccb_linear_backward_get_workspace_size", a)[1]
    return run("mccb_linear_backward", a, go, go_ld, pre, gx, gw, gb, ws, wsz, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), NULLPTR), (dict(weight=None), NULLPTR), (dict(out=None), NULLPTR),
    (dict(dtype=3), INVALID), (dict(activation=5), INVALID), (dict(activation=-1), INVALID),
    (dict(M=-1), SHAPE), (dict(N=0), SHAPE), (dict(K=0), SHAPE), (dict(N=1 << 22), SHAPE),
    (dict(x_ld=-64), INVALID), (dict(res_ld=-1), INVALID), (dict(x=ADDR[0] + 1), INVALID),
    (dict(res=ADDR[3] + 1), INVALID), (dict(out=ADDR[0]), INVALID), (dict(out=ADDR[3]), INVALID),
    (dict(pre=ADDR[4] + 32), INVALID), (dict(out=ADDR[2]), INVALID)])
def test_linear_forward_refuses(kw, code):
    assert linear_forward(**kw) == code


def test_linear_forward_needs_its_workspace():
    a = dict(K=8192, x_ld=8192, w_ld=8192)
    rc, need = size("mccb_linear_forward_get_workspace_size", linear(**a))
    assert rc == OK and need > 0  # few tiles and a long contraction: it is split
    assert linear_forward(ws=None, wsz=need, **a) == NULLPTR
    assert linear_forward(wsz=need - 1, **a) == INVALID
    assert linear_forward(ws=ADDR[4], wsz=need, **a) == INVALID


@pytest.mark.parametrize("kw,code", [
    (dict(go=None), NULLPTR), (dict(pre=None), NULLPTR), (dict(x=None), NULLPTR), (dict(ws=None), NULLPTR),
    (dict(wsz=0), INVALID), (dict(ws=ADDR[8] + 2), INVALID), (dict(go_ld=-48), INVALID),
    (dict(gx=ADDR[0]), INVALID), (dict(gw=ADDR[5]), INVALID), (dict(gb=ADDR[4]), INVALID),
    (dict(ws=ADDR[6]), INVALID), (dict(gx=ADDR[5] + 1), INVALID)])
def test_linear_backward_refuses(kw, code):
    assert linear_backward(**kw) == code


@pytest.mark.parametrize("name", sorted(n for n in ssm._SIGNATURES if n.endswith("_size")))
def test_size_calls_refuse_null(name):
    args = {"conv": conv, "scan": scan, "line": linear}[name[5:9]]()
    assert getattr(ssm.ssm_lib(), name)(ctypes.addressof(args), None) == NULLPTR
    out = ctypes.c_uint64(0)
    assert getattr(ssm.ssm_lib(), name)(None, ctypes.addressof(out)) == NULLPTR


# -- the tensor front end, on tensors that it must refuse ---------------------------------------------
def test_front_end_refuses_host_tensors_and_wrong_kinds():
    x, w = torch.zeros((4, 2, 8), dtype=torch.bfloat16), torch.zeros((4, 8), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="HIP device"):
        mdc.conv_act_forward(x, w)
    with pytest.raises(TypeError):
        mdc.conv_act_forward([1.0], w)
    with pytest.raises(ValueError, match="HIP device"):
        mdc.scan_forward(x, x, torch.zeros((4, 8)), x, x)
    with pytest.raises(ValueError, match="HIP device"):
        mdc.linear_forward(x[0], w)
    with pytest.raises(ValueError, match="evenly spaced"):
        mdc.linear_forward(torch.zeros((2, 4, 8), dtype=torch.bfloat16).transpose(0, 1), w)
    with pytest.raises(ValueError, match="contiguous"):
        mdc.linear_forward(torch.zeros((8, 4), dtype=torch.bfloat16).t(), w)
