"""The selective state space block's operators on device tensors: causal convolution with activation
and carried rows, selective scan, and matrix product with its epilogue (``include/mccb_ssm.h``).

Like the rest of the package this layer only checks and marshals arguments (here in ``_ssm``, compiled
from ``csrc/ssm_binding.cpp``); every step of the computation runs in the library's HIP kernels. Data
tensors are time-major ([S,B,...]) and may be strided views; weights and states are contiguous. Calls
enqueue on `stream` (default: torch's current stream) and return without synchronizing. What a call
allocates (outputs that are not given, workspaces) belongs to that stream. Nothing here builds an
autograd graph: each backward is a call of its own.

``ssm_lib()`` is the library itself, for calls of the C-ABI with device addresses; its argument structs are
``ConvArgs``, ``ScanArgs``, ``ScanGradArgs`` and ``LinearArgs``.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import build as _build
from ._lib import bound_module, load, on_stream

ACTIVATIONS = {None: 0, "none": 0, "relu": 1, "silu": 2, "gelu": 3, "softplus": 4}

_i64, _i32, _u64, _vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_uint64, ctypes.c_void_p


def _fields(text):
    """Field list from 'type: name name ...; ...'; name*3 stands for name0 name1 name2."""
    kinds = {"i": _i64, "w": _i32, "f": ctypes.c_float, "p": _vp}
    out = []
    for part in text.split(";"):
        kind, names = part.split(":")
        for name in names.split():
            name, _, n = name.partition("*")
            out += [(name + str(k), kinds[kind.strip()]) for k in range(int(n))] if n else \
                [(name, kinds[kind.strip()])]
    return out


class ConvArgs(ctypes.Structure):
    """mccb_conv_t, its stride arrays as separate fields."""
    _fields_ = _fields("i: S B H W; w: dtype activation; p: x; i: x_stride*3; "
                       "p: weight bias lengths state")


class ScanArgs(ctypes.Structure):
    """mccb_scan_t, its stride arrays as separate fields."""
    _fields_ = _fields("i: S B H N G; w: dtype softplus; p: x dt z Bm Cm; "
                       "i: x_stride*3 dt_stride*3 z_stride*3 b_stride*4 c_stride*4; "
                       "p: A D dt_bias lengths state")


class ScanGradArgs(ctypes.Structure):
    """mccb_scan_grads_t, its stride array as separate fields."""
    _fields_ = _fields("p: gradOut; i: gout_stride*3; p: gradFinalState gradX gradDt gradZ gradB "
                       "gradC gradA gradD gradDtBias gradState")


class LinearArgs(ctypes.Structure):
    """mccb_linear_t."""
    _fields_ = _fields("i: M K N; w: dtype activation; p: x weight bias; i: x_ld weight_ld; "
                       "w: pre_fp32")


_SIGNATURES = {
    "mccb_conv_act_forward": (ConvArgs, _vp, _vp, _vp),
    "mccb_conv_act_backward_get_workspace_size": (ConvArgs, _vp),
    "mccb_conv_act_backward": (ConvArgs, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _u64, _vp),
    "mccb_conv_act_step": (ConvArgs, _vp, _vp, _vp),
    "mccb_scan_saved_size": (ScanArgs, _vp),
    "mccb_scan_forward_get_workspace_size": (ScanArgs, _vp),
    "mccb_scan_forward": (ScanArgs, _vp, _vp, _vp, _vp, _u64, _vp),
    "mccb_scan_backward_get_workspace_size": (ScanArgs, _vp),
    "mccb_scan_backward": (ScanArgs, _vp, _vp, _vp, _u64, _vp),
    "mccb_scan_step": (ScanArgs, _vp, _vp, _vp),
    "mccb_linear_forward_get_workspace_size": (LinearArgs, _vp),
    "mccb_linear_forward": (LinearArgs, _vp, _i64, _vp, _vp, _vp, _u64, _vp),
    "mccb_linear_backward_get_workspace_size": (LinearArgs, _vp),
    "mccb_linear_backward": (LinearArgs, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _u64, _vp),
}

_lib = None
_module = None


def ssm_lib() -> ctypes.CDLL:
    """The loaded library of these operators, built first if no build exists."""
    global _lib
    if _lib is None:
        L = load(_build.SSM_LIB, "MCCB_SSM_LIBRARY", _build.build_ssm_library)
        for name, sig in _SIGNATURES.items():
            f = getattr(L, name)
            f.argtypes = [_vp, *sig[1:]]  # the argument struct by address
            f.restype = ctypes.c_int
        _lib = L
    return _lib


def ssm_module():
    """The compiled front end, bound to the library; built first if no build exists."""
    global _module
    if _module is None:
        _module = bound_module("_ssm", _build.BINDING, _build.build_binding, ssm_lib(), _SIGNATURES)
    return _module


def _activation(name, allowed):
    code = ACTIVATIONS.get(name)
    if code is None or code not in allowed:
        raise ValueError(f"activation {name!r} not supported here")
    return code


def _call(function, stream, *args):
    """function(*args) of the front end, on `stream` if one is given."""
    if stream is None:
        return getattr(_module or ssm_module(), function)(*args)
    return on_stream(getattr(_module or ssm_module(), function), stream, args)


# -- causal convolution with activation and carried rows ---------------------------------------------
class ConvGrads(NamedTuple):
    x: torch.Tensor
    weight: torch.Tensor
    bias: Optional[torch.Tensor]
    state: Optional[torch.Tensor]


def conv_act_forward(x, weight, bias=None, activation="silu", lengths=None, state=None,
                     return_state=False, y=None, final_state=None, stream=None):
    """y [S,B,H] = activation(bias + causal depthwise conv(x, weight)); x [S,B,H], weight [W,H]
    (W = 1..4), bias [H], activation "silu" or None.

    `state` [W-1,B,H] holds the rows before the first (zeros if None). With `return_state` the
    result is (y, final_state), the last W-1 rows before each sequence's end, to go on from. Rows
    at or past `lengths` (int64 [B] on the device) give zeros and are not computed with."""
    return _call("conv_forward", stream, x, weight, bias, _activation(activation, (0, 2)), lengths,
                 state, bool(return_state), y, final_state)


def conv_act_backward(gradY, x, weight, bias=None, activation="silu", lengths=None, state=None,
                      gradFinalState=None, stream=None) -> ConvGrads:
    """Gradients of conv_act_forward with the same arguments: of x [S,B,H], of weight [W,H], of bias
    and of state where those were given. gradY [S,B,H] may be strided; gradFinalState [W-1,B,H]
    is the gradient of the returned state, if one flows back."""
    return ConvGrads(*_call("conv_backward", stream, gradY, x, weight, bias,
                            _activation(activation, (0, 2)), lengths, state, gradFinalState))


def conv_act_step(x, weight, state, bias=None, activation="silu", y=None, stream=None):
    """One token: y [B,H] from x [B,H] and the carried rows `state` [W-1,B,H], which are moved up by
    one in place."""
    return _call("conv_step", stream, x, weight, state, bias, _activation(activation, (0, 2)), y)


# -- selective scan ----------------------------------------------------------------------------------
class ScanGrads(NamedTuple):
    x: torch.Tensor
    dt: torch.Tensor
    A: torch.Tensor
    B: torch.Tensor
    C: torch.Tensor
    D: Optional[torch.Tensor]
    z: Optional[torch.Tensor]
    dt_bias: Optional[torch.Tensor]
    state: Optional[torch.Tensor]


def scan_forward(x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus=True, lengths=None,
                 state=None, return_state=False, return_saved=False, out=None, final_state=None,
                 stream=None):
    """Selective state space scan over x, dt, z [S,B,H] with A [N,H] fp32 (N = 1..32), B and C
    [S,B,G,N] (or [S,B,N] for one group), D and dt_bias [H] fp32; out [S,B,H].

    `state` [B,N,H] fp32 is the state before the first row (zeros if None). The result is out, or
    a tuple of it with the state after each sequence's last row (`return_state`) and what
    scan_backward needs (`return_saved`). Rows at or past `lengths` (int64 [B] on the device) give
    zeros and leave the state alone."""
    return _call("scan_forward", stream, x, dt, A, B, C, D, z, dt_bias, bool(softplus), lengths, state,
                 bool(return_state), bool(return_saved), out, final_state)


def scan_backward(gradOut, x, dt, A, B, C, saved, D=None, z=None, dt_bias=None, softplus=True,
                  lengths=None, state=None, gradFinalState=None, stream=None) -> ScanGrads:
    """Gradients of scan_forward with the same arguments and what it saved: of every input that was
    given. gradOut [S,B,H] may be strided; gradFinalState [B,N,H] fp32 is the gradient of the
    returned state, if one flows back."""
    return ScanGrads(*_call("scan_backward", stream, x, dt, A, B, C, D, z, dt_bias, bool(softplus),
                            lengths, state, gradOut, saved, gradFinalState))


def scan_step(state, x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus=True, out=None,
              stream=None):
    """One token: out [B,H] from x, dt, z [B,H], B and C [B,G,N] or [B,N]; `state` [B,N,H] fp32 is
    updated in place."""
    return _call("scan_step", stream, x, dt, A, B, C, D, z, dt_bias, bool(softplus), state, out)


# -- matrix product with its epilogue ----------------------------------------------------------------
class LinearGrads(NamedTuple):
    x: Optional[torch.Tensor]
    weight: Optional[torch.Tensor]
    bias: Optional[torch.Tensor]


def linear_forward(x, weight, bias=None, activation=None, residual=None, return_pre=False, out=None,
                   stream=None, pre_dtype=None):
    """out [...,N] = activation(x weight^T + bias) + residual; x [...,K], weight [N,K], bias [N],
    residual [...,N], activation None, "relu", "silu", "gelu" (tanh form) or "softplus". The rows of
    x and residual are contiguous and evenly spaced. With `return_pre` the result is (out, pre),
    pre = x weight^T + bias as linear_backward needs it, in `pre_dtype`: x's (the default) or
    torch.float32, which twice as many bytes keep from rounding."""
    if pre_dtype is not None and pre_dtype not in (torch.float32, x.dtype):
        raise ValueError(f"pre_dtype {pre_dtype} not supported (x's dtype, float32)")
    return _call("linear_forward", stream, x, weight, bias, _activation(activation, (0, 1, 2, 3, 4)),
                 residual, bool(return_pre), out, pre_dtype == torch.float32)


def linear_backward(gradOut, x, weight, pre=None, activation=None, grad_x=True, grad_weight=True,
                    grad_bias=True, stream=None) -> LinearGrads:
    """Gradients of linear_forward for gradOut [...,N]: of x, weight and bias, as asked for. `pre` is
    linear_forward's, in either type (not needed without an activation): the activation's slope is
    taken at it as it was rounded. gradOut times that slope is rounded to gradOut's type for the
    products. The residual's gradient is gradOut."""
    return LinearGrads(*_call("linear_backward", stream, gradOut, x, weight, pre,
                              _activation(activation, (0, 1, 2, 3, 4)), bool(grad_x),
                              bool(grad_weight), bool(grad_bias)))
