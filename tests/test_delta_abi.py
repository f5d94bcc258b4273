"""The C-ABI of the delta rule and the norms without a GPU: exports, struct sizes, workspace sizes, refusals. Every
call that passes made-up addresses is one that the host-side checks must reject before any HIP call."""
from __future__ import annotations

import ctypes
import os
import re
import subprocess

import pytest
import torch

import masked_depthwise_causal_amd as mdc
from masked_depthwise_causal_amd import build as mbuild
from masked_depthwise_causal_amd import delta

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mccb_delta.h")
OK, NULLPTR, INVALID, SHAPE = mdc.MCCB_OK, mdc.MCCB_ERR_PARAM_NULLPTR, mdc.MCCB_ERR_PARAM_INVALID, mdc.MCCB_ERR_SHAPE
GB = 1 << 30
ADDR = [0x7E0000000000 + k * 16 * GB for k in range(28)]  # never dereferenced


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(mccb_[a-z_]+)\s*\(", text)))


def test_exports_every_declared_function():
    lib = delta.delta_lib()
    assert set(declared()) == set(delta._SIGNATURES)
    out = subprocess.run(["nm", "-D", "--defined-only", mbuild.DELTA_LIB], capture_output=True, text=True,
                         check=True).stdout
    assert set(declared()) <= set(re.findall(r"\bT (mccb_\w+)", out))
    assert all(hasattr(lib, n) for n in declared())


def test_struct_sizes_match_the_header(tmp_path):
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include "mccb_delta.h"\nint main(void) { printf("%zu %zu %zu", '
                   "sizeof(mccb_delta_t), sizeof(mccb_delta_grads_t), sizeof(mccb_norm_t)); return 0; }\n")
    exe = str(tmp_path / "sizes")
    subprocess.run(["gcc", "-std=c11", "-I", mbuild.INCLUDE, str(src), "-o", exe], check=True)
    got = [int(v) for v in subprocess.run([exe], capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(t) for t in (delta.DeltaArgs, delta.DeltaGradArgs, delta.NormArgs)]


def run(name, args, *rest):
    rc = getattr(delta.delta_lib(), name)(ctypes.addressof(args) if args is not None else None, *rest)
    assert rc != OK, f"{name} passed its checks with made-up addresses"
    return rc


def size(name, args):
    out = ctypes.c_uint64(0)
    rc = getattr(delta.delta_lib(), name)(ctypes.addressof(args), ctypes.addressof(out))
    return rc, out.value


# -- delta rule ----------------------------------------------------------------------------------------
def args(S=70, B=2, H=4, G=2, K=16, V=24, dtype=0, softplus=1, normalize=1, scale=0.25, q=ADDR[0], k=ADDR[1], v=ADDR[2],
         dt=ADDR[3], b=ADDR[4], key=(64, 32, 16), val=(192, 96, 24), row=(8, 4, 1), A=ADDR[5], bias=ADDR[6],
         lengths=ADDR[7], state=ADDR[8]):
    return delta.DeltaArgs(S, B, H, G, K, V, dtype, softplus, normalize, scale, q, k, v, dt, b, *key, *key, *val, *row,
                           *row, A, bias, lengths, state)


def forward(out=ADDR[9], final=ADDR[10], saved=None, ws=ADDR[11], wsz=1 << 30, **kw):
    return run("mccb_delta_forward", args(**kw), out, final, saved, ws, wsz, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), NULLPTR), (dict(k=None), NULLPTR), (dict(v=None), NULLPTR), (dict(dt=None), NULLPTR),
    (dict(b=None), NULLPTR), (dict(A=None), NULLPTR), (dict(out=None), NULLPTR), (dict(ws=None), NULLPTR),
    (dict(dtype=2), INVALID), (dict(S=-1), SHAPE), (dict(S=1 << 28), SHAPE), (dict(B=0), SHAPE), (dict(H=0), SHAPE),
    (dict(G=3), SHAPE), (dict(G=0), SHAPE), (dict(G=8), SHAPE), (dict(K=0), SHAPE), (dict(K=129), SHAPE),
    (dict(V=0), SHAPE), (dict(V=257), SHAPE), (dict(B=256, H=256), SHAPE), (dict(B=1 << 40, H=1 << 40), SHAPE),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(wsz=100), INVALID),
    (dict(ws=ADDR[11] + 8), INVALID), (dict(key=(-64, 32, 16)), INVALID), (dict(val=(1 << 62, 96, 24)), INVALID),
    (dict(q=ADDR[0] + 1), INVALID), (dict(A=ADDR[5] + 2), INVALID), (dict(lengths=ADDR[7] + 4), INVALID),
    (dict(state=ADDR[8] + 2), INVALID), (dict(out=ADDR[9] + 1), INVALID), (dict(final=ADDR[10] + 2), INVALID),
    (dict(out=ADDR[2]), INVALID), (dict(final=ADDR[8]), INVALID), (dict(final=ADDR[9] + 64), INVALID),
    (dict(ws=ADDR[0]), INVALID), (dict(saved=ADDR[12] + 8), INVALID), (dict(saved=ADDR[1]), INVALID)])
def test_delta_forward_refuses(kw, code):
    assert forward(**kw) == code


GRADS = dict(go=ADDR[12], gfinal=ADDR[13], gq=ADDR[14], gk=ADDR[15], gv=ADDR[16], gdt=ADDR[17], gb=ADDR[18], gA=ADDR[19],
             gbias=ADDR[20], gstate=ADDR[21])


def backward(saved=ADDR[22], ws=ADDR[23], wsz=None, gstride=(192, 96, 24), **kw):
    g = {**GRADS, **{n: kw.pop(n) for n in list(kw) if n in GRADS}}
    a = args(**kw)
    if wsz is None:
        wsz = size("mccb_delta_backward_get_workspace_size", a)[1]
    ga = delta.DeltaGradArgs(g["go"], *gstride, g["gfinal"], *(g[n] for n in ("gq", "gk", "gv", "gdt", "gb", "gA",
                                                                              "gbias", "gstate")))
    return run("mccb_delta_backward", a, ctypes.addressof(ga), saved, ws, wsz, None)


@pytest.mark.parametrize("kw,code", [
    (dict(go=None), NULLPTR), (dict(gq=None), NULLPTR), (dict(gk=None), NULLPTR), (dict(gv=None), NULLPTR),
    (dict(gdt=None), NULLPTR), (dict(gb=None), NULLPTR), (dict(gA=None), NULLPTR), (dict(saved=None), NULLPTR),
    (dict(ws=None), NULLPTR), (dict(wsz=64), INVALID), (dict(ws=ADDR[23] + 4), INVALID), (dict(saved=ADDR[22] + 4), INVALID),
    (dict(gstride=(192, -1, 24)), INVALID), (dict(gq=ADDR[0]), INVALID), (dict(gk=ADDR[14]), INVALID),
    (dict(gstate=ADDR[13]), INVALID), (dict(gv=ADDR[12]), INVALID), (dict(gA=ADDR[19] + 2), INVALID),
    (dict(gb=ADDR[18] + 1), INVALID), (dict(ws=ADDR[22]), INVALID), (dict(K=200), SHAPE)])
def test_delta_backward_refuses(kw, code):
    assert backward(**kw) == code


def test_delta_backward_refuses_no_gradients():
    assert run("mccb_delta_backward", args(), None, ADDR[22], ADDR[23], 1 << 30, None) == NULLPTR


@pytest.mark.parametrize("kw,state,out,code", [
    (dict(), None, ADDR[9], NULLPTR), (dict(), ADDR[10], None, NULLPTR), (dict(S=2), ADDR[10], ADDR[9], SHAPE),
    (dict(lengths=ADDR[7]), ADDR[10], ADDR[9], INVALID), (dict(state=ADDR[8]), ADDR[10], ADDR[9], INVALID),
    (dict(), ADDR[10], ADDR[10], INVALID), (dict(), ADDR[0], ADDR[9], INVALID), (dict(), ADDR[10] + 2, ADDR[9], INVALID)])
def test_delta_step_refuses(kw, state, out, code):
    a = args(**{"S": 1, "lengths": None, "state": None, **kw})
    assert run("mccb_delta_step", a, state, out, None) == code


def test_sizes_grow_with_what_is_kept():
    one, two = (size("mccb_delta_saved_size", args(S=s))[1] for s in (64, 65))
    assert two == 2 * one  # whole chunks of 64 rows
    assert size("mccb_delta_forward_get_workspace_size", args(S=0)) == (OK, 0)
    assert size("mccb_delta_forward_get_workspace_size", args())[1] < size("mccb_delta_saved_size", args())[1]
    # the largest sizes that are taken do not overflow
    rc, n = size("mccb_delta_saved_size", args(S=(1 << 28) - 1, B=65535, H=1, G=1, K=128, V=256))
    assert rc == OK and n > (1 << 50)


# -- norms ---------------------------------------------------------------------------------------------
def norm(R=6, H=24, groups=1, dtype=0, shared=0, eps=1e-6, x=ADDR[0], w=ADDR[1], residual=ADDR[2], scale=ADDR[3], z=None,
         x_ld=24, residual_ld=24, z_ld=24):
    return delta.NormArgs(R, H, groups, dtype, shared, eps, x, w, residual, scale, z, x_ld, residual_ld, z_ld)


NORM = [(dict(x=None), NULLPTR), (dict(w=None), NULLPTR), (dict(dtype=3), INVALID), (dict(R=-1), SHAPE),
        (dict(R=1 << 31), SHAPE), (dict(H=0), SHAPE), (dict(H=16385), SHAPE), (dict(eps=0.0), INVALID),
        (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(x_ld=-1), INVALID), (dict(x=ADDR[0] + 1), INVALID),
        (dict(w=ADDR[1] + 1), INVALID), (dict(out=None), NULLPTR), (dict(out=ADDR[4] + 1), INVALID), (dict(out=ADDR[0]), INVALID),
        (dict(out=ADDR[2] + 16), INVALID)]


@pytest.mark.parametrize("kw,code", NORM + [(dict(groups=2), INVALID), (dict(z=ADDR[5]), INVALID), (dict(total=ADDR[4]), INVALID)])
def test_prenorm_forward_refuses(kw, code):
    kw = dict(kw)
    out, total = kw.pop("out", ADDR[4]), kw.pop("total", ADDR[6])
    assert run("mccb_prenorm_forward", norm(**kw), out, total, None) == code


@pytest.mark.parametrize("kw,code", NORM + [(dict(groups=5), SHAPE), (dict(groups=0), SHAPE), (dict(z=ADDR[5] + 1), INVALID)])
def test_postnorm_forward_refuses(kw, code):
    kw = dict(kw)
    out = kw.pop("out", ADDR[4])
    assert run("mccb_postnorm_forward", norm(**kw), out, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(go=None), NULLPTR), (dict(gx=None), NULLPTR), (dict(gw=None), NULLPTR), (dict(gscale=None), NULLPTR),
    (dict(ws=None), NULLPTR), (dict(wsz=1), INVALID), (dict(ws=ADDR[10] + 8), INVALID), (dict(gx=ADDR[0]), INVALID),
    (dict(gres=ADDR[5]), INVALID), (dict(residual=None), INVALID), (dict(scale=None), INVALID), (dict(go_ld=-4), INVALID),
    (dict(gw=ADDR[7] + 1), INVALID)])
def test_prenorm_backward_refuses(kw, code):
    p = dict(go=ADDR[4], go_ld=24, gsum=ADDR[5], gx=ADDR[6], gres=ADDR[9], gw=ADDR[7], gscale=ADDR[8], ws=ADDR[10], wsz=None)
    p.update({n: kw[n] for n in kw if n in p})
    a = norm(**{n: v for n, v in kw.items() if n not in p})
    if p["wsz"] is None:
        p["wsz"] = size("mccb_prenorm_backward_get_workspace_size", a)[1]
    assert run("mccb_prenorm_backward", a, p["go"], p["go_ld"], p["gsum"], 24, p["gx"], p["gres"], p["gw"], p["gscale"],
               p["ws"], p["wsz"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(gz=None), NULLPTR), (dict(z=None), INVALID), (dict(gz=ADDR[6]), INVALID), (dict(ws=ADDR[5]), INVALID)])
def test_postnorm_backward_refuses(kw, code):
    a = norm(groups=2, residual=None, z=kw.get("z", ADDR[5]))
    wsz = size("mccb_postnorm_backward_get_workspace_size", a)[1]
    assert run("mccb_postnorm_backward", a, ADDR[4], 24, ADDR[6], kw.get("gz", ADDR[9]), ADDR[7], ADDR[8],
               kw.get("ws", ADDR[10]), wsz, None) == code


@pytest.mark.parametrize("name", sorted(n for n in delta._SIGNATURES if n.endswith("_size")))
def test_size_calls_refuse_null(name):
    a = args() if "delta" in name else norm()
    assert getattr(delta.delta_lib(), name)(ctypes.addressof(a), None) == NULLPTR
    out = ctypes.c_uint64(0)
    assert getattr(delta.delta_lib(), name)(None, ctypes.addressof(out)) == NULLPTR


def test_front_end_refuses_host_tensors_and_wrong_kinds():
    x, w = torch.zeros((4, 8), dtype=torch.bfloat16), torch.zeros(8, dtype=torch.bfloat16)
    q, v, d = (torch.zeros(s, dtype=torch.bfloat16) for s in ((4, 2, 1, 8), (4, 2, 1, 8), (4, 2, 1)))
    with pytest.raises(ValueError, match="HIP device"):
        mdc.prenorm_forward(x, w)
    with pytest.raises(ValueError, match="HIP device"):
        mdc.postnorm_forward(x, w)
    with pytest.raises(TypeError):
        mdc.prenorm_forward(3.0, w)
    with pytest.raises(ValueError, match="HIP device"):
        mdc.delta_forward(q, q, v, d, d, torch.zeros(1))
    with pytest.raises(ValueError, match="HIP device"):
        mdc.delta_step(torch.zeros((2, 1, 8, 8)), q[0], q[0], v[0], d[0], d[0], torch.zeros(1))
    with pytest.raises(TypeError):
        mdc.delta_forward([1.0], q, v, d, d, torch.zeros(1))

    class Stream:
        device = torch.device("cuda", 1)

    with pytest.raises(ValueError, match="stream lives on cuda:1"):
        mdc.prenorm_forward(x, w, stream=Stream())


def test_flags_are_read_before_anything_runs():
    q, v, d, flag = torch.zeros((4, 2, 1, 8)), torch.zeros((4, 2, 1, 8)), torch.zeros((4, 2, 1)), torch.zeros(2)
    for kw in ({"softplus": flag}, {"normalize": flag}, {"return_state": flag}):
        with pytest.raises(RuntimeError, match="Boolean value"):
            mdc.delta_forward(q, q, v, d, d, torch.zeros(1), **kw)
    with pytest.raises((TypeError, ValueError)):
        mdc.prenorm_forward(q, d, eps="small")
