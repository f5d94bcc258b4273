"""The gated delta rule and the norms before and after a block, on device tensors
(``include/mccb_delta.h``).

As in ``ssm`` this layer only checks and marshals arguments (in ``_delta``, compiled from
``csrc/delta_binding.cpp``); every step of the computation runs in the library's HIP kernels. Calls enqueue on
`stream` (default: torch's current stream) and return without synchronizing. What a call allocates
(outputs that are not given, workspaces) belongs to that stream. Nothing here builds an autograd graph: each
backward is a call of its own.

``delta_lib()`` is the library itself, for calls of the C-ABI with device addresses; its argument structs are
``DeltaArgs``, ``DeltaGradArgs`` and ``NormArgs``.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import build as _build
from ._lib import bound_module, load, on_stream
from .ssm import _fields

_i64, _u64, _vp = ctypes.c_int64, ctypes.c_uint64, ctypes.c_void_p


class DeltaArgs(ctypes.Structure):
    """mccb_delta_t, its stride arrays as separate fields."""
    _fields_ = _fields("i: S B H G K V; w: dtype softplus normalize; f: scale; p: q k v dt b; "
                       "i: q_stride*3 k_stride*3 v_stride*3 dt_stride*3 b_stride*3; "
                       "p: A dt_bias lengths state")


class DeltaGradArgs(ctypes.Structure):
    """mccb_delta_grads_t, its stride array as separate fields."""
    _fields_ = _fields("p: gradOut; i: gout_stride*3; p: gradFinalState gradQ gradK gradV gradDt gradB "
                       "gradA gradDtBias gradState")


class NormArgs(ctypes.Structure):
    """mccb_norm_t."""
    _fields_ = _fields("i: R H groups; w: dtype weight_shared; f: eps; p: x weight residual scale z; "
                       "i: x_ld residual_ld z_ld")


_SIGNATURES = {
    "mccb_delta_saved_size": (DeltaArgs, _vp),
    "mccb_delta_forward_get_workspace_size": (DeltaArgs, _vp),
    "mccb_delta_forward": (DeltaArgs, _vp, _vp, _vp, _vp, _u64, _vp),
    "mccb_delta_backward_get_workspace_size": (DeltaArgs, _vp),
    "mccb_delta_backward": (DeltaArgs, _vp, _vp, _vp, _u64, _vp),
    "mccb_delta_step": (DeltaArgs, _vp, _vp, _vp),
    "mccb_prenorm_forward": (NormArgs, _vp, _vp, _vp),
    "mccb_prenorm_backward_get_workspace_size": (NormArgs, _vp),
    "mccb_prenorm_backward": (NormArgs, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _u64, _vp),
    "mccb_postnorm_forward": (NormArgs, _vp, _vp),
    "mccb_postnorm_backward_get_workspace_size": (NormArgs, _vp),
    "mccb_postnorm_backward": (NormArgs, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _u64, _vp),
}

_lib = None
_module = None


def delta_lib() -> ctypes.CDLL:
    """The loaded library of these operators, built first if no build exists."""
    global _lib
    if _lib is None:
        L = load(_build.DELTA_LIB, "MCCB_DELTA_LIBRARY", _build.build_delta_library)
        for name, sig in _SIGNATURES.items():
            f = getattr(L, name)
            f.argtypes = [_vp, *sig[1:]]  # the argument struct by address
            f.restype = ctypes.c_int
        _lib = L
    return _lib


def delta_module():
    """The compiled front end, bound to the library; built first if no build exists."""
    global _module
    if _module is None:
        _module = bound_module("_delta", _build.DELTA_BINDING, _build.build_delta_binding, delta_lib(),
                               _SIGNATURES)
    return _module


def _call(function, stream, *args):
    """function(*args) of the front end, on `stream` if one is given."""
    f = getattr(_module or delta_module(), function)
    return f(*args) if stream is None else on_stream(f, stream, args)


# -- gated delta rule --------------------------------------------------------------------------------
class DeltaGrads(NamedTuple):
    q: torch.Tensor
    k: torch.Tensor
    v: torch.Tensor
    dt: torch.Tensor
    b: torch.Tensor
    A: torch.Tensor
    dt_bias: Optional[torch.Tensor]
    state: Optional[torch.Tensor]


def delta_forward(q, k, v, dt, b, A, dt_bias=None, softplus=True, normalize=True, scale=None, lengths=None,
                  state=None, return_state=False, return_saved=False, out=None, final_state=None,
                  stream=None):
    """Gated delta rule over q, k [S,B,G,K] (K up to 128), v [S,B,H,V] (V up to 256), dt and b [S,B,H], with
    A and dt_bias [H] fp32; out [S,B,H,V]. H is a multiple of G: value head h has key head h // (H // G).

    Row by row, for a head's state S [K,V]: a = exp(A softplus(dt + dt_bias)), beta = sigmoid(b),
    u = beta (v - a S^T k), S = a S + k u^T, out = scale S^T q, with q and k divided by their norms unless
    `normalize` is False; scale is K ** -0.5 unless given. q, k and v have contiguous rows.

    `state` [B,H,K,V] fp32 is the state before the first row (zeros if None). The result is out, or a tuple
    of it with the state after each sequence's last row (`return_state`) and what delta_backward needs
    (`return_saved`). Rows at or past `lengths` (int64 [B] on the device) give zeros and leave the state
    alone. Computed in chunks of 64 rows with products of about 22 bits and fp32 sums (mccb_delta.h)."""
    return _call("delta_forward", stream, q, k, v, dt, b, A, dt_bias, bool(softplus), bool(normalize),
                 None if scale is None else float(scale), lengths, state, bool(return_state),
                 bool(return_saved), out, final_state)


def delta_backward(gradOut, q, k, v, dt, b, A, saved, dt_bias=None, softplus=True, normalize=True, scale=None,
                   lengths=None, state=None, gradFinalState=None, stream=None) -> DeltaGrads:
    """Gradients of delta_forward with the same arguments and what it saved: of every input that was
    given. gradOut [S,B,H,V] may be strided, with contiguous rows; gradFinalState [B,H,K,V] fp32 is the
    gradient of the returned state, if one flows back."""
    return DeltaGrads(*_call("delta_backward", stream, q, k, v, dt, b, A, dt_bias, bool(softplus),
                             bool(normalize), None if scale is None else float(scale), lengths, state,
                             gradOut, saved, gradFinalState))


def delta_step(state, q, k, v, dt, b, A, dt_bias=None, softplus=True, normalize=True, scale=None, out=None,
               stream=None):
    """One token: out [B,H,V] from q, k [B,G,K], v [B,H,V], dt and b [B,H]; `state` [B,H,K,V] fp32 is
    updated in place."""
    return _call("delta_step", stream, q, k, v, dt, b, A, dt_bias, bool(softplus), bool(normalize),
                 None if scale is None else float(scale), state, out)


# -- norms before and after a block ------------------------------------------------------------------
class PrenormGrads(NamedTuple):
    x: torch.Tensor
    weight: torch.Tensor
    residual: Optional[torch.Tensor]
    scale: Optional[torch.Tensor]


class PostnormGrads(NamedTuple):
    x: torch.Tensor
    weight: torch.Tensor
    z: Optional[torch.Tensor]
    scale: Optional[torch.Tensor]


def prenorm_forward(x, weight, residual=None, scale=None, eps=1e-6, return_sum=False, out=None,
                    sum_out=None, stream=None):
    """out [...,H] = sum / sqrt(mean(sum^2) + eps) * weight, with sum = residual + scale * x; x and residual
    [...,H] of evenly spaced, contiguous rows, weight and scale [H], H up to 16384. With `return_sum` the
    result is (out, sum), to add the next block's output to; where neither residual nor scale is given
    that sum is x itself (unless `sum_out` asks for a copy). The norm is of the sum before its rounding."""
    return _call("prenorm_forward", stream, x, weight, residual, scale, float(eps), bool(return_sum), out,
                 sum_out)


def prenorm_backward(gradOut, x, weight, residual=None, scale=None, eps=1e-6, gradSum=None,
                     stream=None) -> PrenormGrads:
    """Gradients of prenorm_forward with the same arguments: of x, weight, and residual and scale where
    those were given. gradSum [...,H] is the gradient that reaches the sum from elsewhere, as from the
    next addition. Without a scale the residual's gradient is x's, the same tensor."""
    return PrenormGrads(*_call("prenorm_backward", stream, gradOut, x, weight, residual, scale, float(eps),
                               gradSum))


def postnorm_forward(x, weight, z=None, residual=None, scale=None, groups=1, eps=1e-6, out=None,
                     stream=None):
    """out [...,H] = residual + scale * (x / sqrt(mean(x^2) + eps) * weight * silu(z)), the mean over each
    of `groups` equal parts of a row (up to 16384 values); x, z and residual [...,H] of evenly spaced,
    contiguous rows, scale [H], weight [H], or [H/groups] for a weight that all groups share. z, residual
    and scale may be left out."""
    return _call("postnorm_forward", stream, x, weight, z, residual, scale, int(groups), float(eps), out)


def postnorm_backward(gradOut, x, weight, z=None, scale=None, groups=1, eps=1e-6,
                      stream=None) -> PostnormGrads:
    """Gradients of postnorm_forward with the same arguments: of x, weight, and z and scale where those
    were given. The residual's gradient is gradOut."""
    return PostnormGrads(*_call("postnorm_backward", stream, gradOut, x, weight, z, scale, int(groups),
                                float(eps)))
