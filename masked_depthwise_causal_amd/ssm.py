"""The selective state space block's operators on device tensors: causal convolution with activation
and carried rows, selective scan, and matrix product with its epilogue (``include/mccb_ssm.h``).

Like the rest of the package this layer only checks and marshals arguments; every step of the
computation runs in the library's HIP kernels. Data tensors are time-major ([S,B,...]) and may be
strided views; weights and states are contiguous. Calls enqueue on `stream` (default: torch's current
stream) and return without synchronizing. Outputs are allocated unless given. Nothing here builds
an autograd graph: each backward is a call of its own.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import NamedTuple, Optional

import torch

from . import build as _build
from ._lib import MccbError, load

_OK = 0
_address = ctypes.addressof
_DTYPE = {torch.bfloat16: 0, torch.float16: 1}
ACTIVATIONS = {None: 0, "none": 0, "relu": 1, "silu": 2, "gelu": 3, "softplus": 4}

_i64, _i32, _u64, _vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_uint64, ctypes.c_void_p


def _fields(text):
    """Field list from 'type: name name ...; ...'; name*3 stands for name0 name1 name2."""
    kinds = {"i": _i64, "w": _i32, "p": _vp}
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
    _fields_ = _fields("i: M K N; w: dtype activation; p: x weight bias; i: x_ld weight_ld")


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


# -- argument checks ---------------------------------------------------------------------------------
def _check(name, t, shape, dtype, device, contiguous=False):
    try:
        if t.shape == shape and t.dtype is dtype and t.get_device() == device.index and \
                not (contiguous and not t.is_contiguous()):
            return
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} must live on {device} (a HIP device)")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    raise ValueError(f"{name} must be contiguous")


def _data(name, t, dims):
    """dtype code and device of the tensor that sets them for a call."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must live on a HIP device")
    if t.dim() != len(dims):
        raise ValueError(f"{name} must be [{','.join(dims)}]")
    code = _DTYPE.get(t.dtype)
    if code is None:
        raise ValueError(f"dtype {t.dtype} not supported (bfloat16, float16)")
    return code, t.device


def _activation(name, allowed):
    code = ACTIVATIONS.get(name)
    if code is None or code not in allowed:
        raise ValueError(f"activation {name!r} not supported here")
    return code


def _ptr(t):
    return None if t is None else t.data_ptr()


# The handle of torch's current stream, without the Stream object around it (2 us of a 6 us call).
_current = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _handle(stream, device):
    if stream is not None:
        return stream.cuda_stream
    if _current is not None:
        return _current(device.index)
    return torch.cuda.current_stream(device).cuda_stream


_here = contextlib.nullcontext()


def _On(stream):
    """What a call allocates belongs to the stream that its kernels run on."""
    return _here if stream is None else torch.cuda.stream(stream)


def _size(name, args):
    out = _u64(0)
    rc = getattr(ssm_lib(), name)(ctypes.addressof(args), ctypes.addressof(out))
    if rc != _OK:
        raise MccbError(rc, name)
    return out.value


def _workspace(name, args, device):
    n = _size(name, args)
    return (torch.empty(n, dtype=torch.uint8, device=device), n) if n else (None, 0)


def _run(name, args, *rest):
    rc = getattr(_lib or ssm_lib(), name)(_address(args), *rest)
    if rc != _OK:
        raise MccbError(rc, name)


# -- causal convolution with activation and carried rows ---------------------------------------------
class ConvGrads(NamedTuple):
    x: torch.Tensor
    weight: torch.Tensor
    bias: Optional[torch.Tensor]
    state: Optional[torch.Tensor]


def _conv_args(x, weight, bias, activation, lengths, state):
    code, dev = _data("x", x, "SBH")
    S, B, H = x.shape
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be a [W,H] tensor")
    W = weight.shape[0]
    dt = x.dtype
    _check("weight", weight, (W, H), dt, dev, True)
    if bias is not None:
        _check("bias", bias, (H,), dt, dev, True)
    if lengths is not None:
        _check("lengths", lengths, (B,), torch.int64, dev, True)
    if state is not None:
        _check("state", state, (W - 1, B, H), dt, dev, True)
    return ConvArgs(S, B, H, W, code, _activation(activation, (0, 2)), x.data_ptr(), *x.stride(),
                    weight.data_ptr(), _ptr(bias), _ptr(lengths), _ptr(state)), (S, B, H, W, dt, dev)


def conv_act_forward(x, weight, bias=None, activation="silu", lengths=None, state=None,
                     return_state=False, y=None, final_state=None, stream=None):
    """y [S,B,H] = activation(bias + causal depthwise conv(x, weight)); x [S,B,H], weight [W,H]
    (W = 1..4), bias [H], activation "silu" or None.

    `state` [W-1,B,H] holds the rows before the first (zeros if None). With `return_state` the
    result is (y, final_state), the last W-1 rows before each sequence's end, to go on from. Rows
    at or past `lengths` (int64 [B] on the device) give zeros and are not computed with."""
    args, (S, B, H, W, dt, dev) = _conv_args(x, weight, bias, activation, lengths, state)
    with _On(stream):
        if y is None:
            y = torch.empty((S, B, H), dtype=dt, device=dev)
        else:
            _check("y", y, (S, B, H), dt, dev, True)
        if final_state is not None:
            _check("final_state", final_state, (W - 1, B, H), dt, dev, True)
        elif return_state:
            final_state = torch.empty((W - 1, B, H), dtype=dt, device=dev)
    _run("mccb_conv_act_forward", args, y.data_ptr(), _ptr(final_state), _handle(stream, dev))
    return (y, final_state) if return_state else y


def conv_act_backward(gradY, x, weight, bias=None, activation="silu", lengths=None, state=None,
                      gradFinalState=None, stream=None) -> ConvGrads:
    """Gradients of conv_act_forward with the same arguments: of x [S,B,H], of weight [W,H], of bias
    and of state where those were given. gradY [S,B,H] may be strided; gradFinalState [W-1,B,H]
    is the gradient of the returned state, if one flows back."""
    args, (S, B, H, W, dt, dev) = _conv_args(x, weight, bias, activation, lengths, state)
    _check("gradY", gradY, (S, B, H), dt, dev)
    if gradFinalState is not None:
        _check("gradFinalState", gradFinalState, (W - 1, B, H), dt, dev, True)
    with _On(stream):
        g = ConvGrads(torch.empty((S, B, H), dtype=dt, device=dev), torch.empty_like(weight),
                      None if bias is None else torch.empty_like(bias),
                      None if state is None else torch.empty_like(state))
        ws, n = _workspace("mccb_conv_act_backward_get_workspace_size", args, dev)
    gs = (_i64 * 3)(*gradY.stride())
    _run("mccb_conv_act_backward", args, gradY.data_ptr(), ctypes.addressof(gs),
         _ptr(gradFinalState), g.x.data_ptr(), g.weight.data_ptr(), _ptr(g.bias), _ptr(g.state),
         _ptr(ws), n, _handle(stream, dev))
    return g


def conv_act_step(x, weight, state, bias=None, activation="silu", y=None, stream=None):
    """One token: y [B,H] from x [B,H] and the carried rows `state` [W-1,B,H], which are moved up by
    one in place."""
    code, dev = _data("x", x, "BH")
    B, H = x.shape
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be a [W,H] tensor")
    W, dt = weight.shape[0], x.dtype
    _check("weight", weight, (W, H), dt, dev, True)
    _check("state", state, (W - 1, B, H), dt, dev, True)
    if bias is not None:
        _check("bias", bias, (H,), dt, dev, True)
    if y is None:
        with _On(stream):
            y = torch.empty((B, H), dtype=dt, device=dev)
    else:
        _check("y", y, (B, H), dt, dev, True)
    args = ConvArgs(1, B, H, W, code, _activation(activation, (0, 2)), x.data_ptr(), 0, *x.stride(),
                    weight.data_ptr(), _ptr(bias))
    _run("mccb_conv_act_step", args, state.data_ptr(), y.data_ptr(), _handle(stream, dev))
    return y


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


_f32 = torch.float32


def _scan_args(x, dt, A, Bm, Cm, D, z, dt_bias, softplus, lengths, state, token=False):
    code, dev = _data("x", x, "BH" if token else "SBH")
    kind, rows = x.dtype, x.shape
    B, H = rows[-2], rows[-1]
    S = 1 if token else rows[0]
    _check("dt", dt, rows, kind, dev)
    if z is not None:
        _check("z", z, rows, kind, dev)
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise ValueError("A must be a [N,H] tensor")
    N = A.shape[0]
    _check("A", A, (N, H), _f32, dev, True)
    if not isinstance(Bm, torch.Tensor) or not isinstance(Cm, torch.Tensor):
        raise TypeError("B and C must be torch.Tensors")
    if Bm.dim() == len(rows):  # one group
        Bm = Bm.unsqueeze(-2)
    if Cm.dim() == len(rows):
        Cm = Cm.unsqueeze(-2)
    if Bm.dim() != len(rows) + 1:
        raise ValueError("B and C must be [S,B,N] or [S,B,G,N] ([B,N] or [B,G,N] for one token)")
    G = Bm.shape[-2]
    _check("B", Bm, (*rows[:-1], G, N), kind, dev)
    _check("C", Cm, (*rows[:-1], G, N), kind, dev)
    if D is not None:
        _check("D", D, (H,), _f32, dev, True)
    if dt_bias is not None:
        _check("dt_bias", dt_bias, (H,), _f32, dev, True)
    if lengths is not None:
        _check("lengths", lengths, (B,), torch.int64, dev, True)
    if state is not None:
        _check("state", state, (B, N, H), _f32, dev, True)
    no_row = (0,) if token else ()
    args = ScanArgs(S, B, H, N, G, code, 1 if softplus else 0, x.data_ptr(), dt.data_ptr(), _ptr(z),
                    Bm.data_ptr(), Cm.data_ptr(), *no_row, *x.stride(), *no_row, *dt.stride(),
                    *((0, 0, 0) if z is None else (*no_row, *z.stride())), *no_row, *Bm.stride(),
                    *no_row, *Cm.stride(), A.data_ptr(), _ptr(D), _ptr(dt_bias), _ptr(lengths),
                    None if token else _ptr(state))
    return args, (S, B, H, N, G, kind, dev)


def scan_forward(x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus=True, lengths=None,
                 state=None, return_state=False, return_saved=False, out=None, final_state=None,
                 stream=None):
    """Selective state space scan over x, dt, z [S,B,H] with A [N,H] fp32 (N = 1..32), B and C
    [S,B,G,N] (or [S,B,N] for one group), D and dt_bias [H] fp32; out [S,B,H].

    `state` [B,N,H] fp32 is the state before the first row (zeros if None). The result is out, or
    a tuple of it with the state after each sequence's last row (`return_state`) and what
    scan_backward needs (`return_saved`). Rows at or past `lengths` (int64 [B] on the device) give
    zeros and leave the state alone."""
    args, (S, Bn, H, N, _, kind, dev) = _scan_args(x, dt, A, B, C, D, z, dt_bias, softplus, lengths,
                                                   state)
    saved = None
    with _On(stream):
        if out is None:
            out = torch.empty((S, Bn, H), dtype=kind, device=dev)
        else:
            _check("out", out, (S, Bn, H), kind, dev, True)
        if final_state is not None:
            _check("final_state", final_state, (Bn, N, H), _f32, dev, True)
        elif return_state:
            final_state = torch.empty((Bn, N, H), dtype=_f32, device=dev)
        if return_saved:
            saved = torch.empty(_size("mccb_scan_saved_size", args) // 4, dtype=_f32, device=dev)
        ws, n = _workspace("mccb_scan_forward_get_workspace_size", args, dev)
    _run("mccb_scan_forward", args, out.data_ptr(), _ptr(final_state), _ptr(saved), _ptr(ws), n,
         _handle(stream, dev))
    if not return_state and not return_saved:
        return out
    return (out,) + ((final_state,) if return_state else ()) + ((saved,) if return_saved else ())


def scan_backward(gradOut, x, dt, A, B, C, saved, D=None, z=None, dt_bias=None, softplus=True,
                  lengths=None, state=None, gradFinalState=None, stream=None) -> ScanGrads:
    """Gradients of scan_forward with the same arguments and what it saved: of every input that was
    given. gradOut [S,B,H] may be strided; gradFinalState [B,N,H] fp32 is the gradient of the
    returned state, if one flows back."""
    args, (S, Bn, H, N, G, kind, dev) = _scan_args(x, dt, A, B, C, D, z, dt_bias, softplus, lengths,
                                                   state)
    _check("gradOut", gradOut, (S, Bn, H), kind, dev)
    _check("saved", saved, (_size("mccb_scan_saved_size", args) // 4,), _f32, dev, True)
    if gradFinalState is not None:
        _check("gradFinalState", gradFinalState, (Bn, N, H), _f32, dev, True)
    with _On(stream):
        def rows(t):
            return torch.empty((S, Bn, H), dtype=kind, device=dev) if t is not None else None

        def like(t):
            return torch.empty_like(t) if t is not None else None

        coef = [torch.empty(t.shape, dtype=kind, device=dev) for t in (B, C)]
        g = ScanGrads(rows(x), rows(dt), like(A), *coef, like(D), rows(z), like(dt_bias),
                      like(state))
        ws, n = _workspace("mccb_scan_backward_get_workspace_size", args, dev)
    grads = ScanGradArgs(gradOut.data_ptr(), *gradOut.stride(), _ptr(gradFinalState),
                         g.x.data_ptr(), g.dt.data_ptr(), _ptr(g.z), g.B.data_ptr(), g.C.data_ptr(),
                         g.A.data_ptr(), _ptr(g.D), _ptr(g.dt_bias), _ptr(g.state))
    _run("mccb_scan_backward", args, ctypes.addressof(grads), _ptr(saved), _ptr(ws), n,
         _handle(stream, dev))
    return g


def scan_step(state, x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus=True, out=None,
              stream=None):
    """One token: out [B,H] from x, dt, z [B,H], B and C [B,G,N] or [B,N]; `state` [B,N,H] fp32 is
    updated in place."""
    args, (_, Bn, H, _, _, kind, dev) = _scan_args(x, dt, A, B, C, D, z, dt_bias, softplus, None,
                                                   state, token=True)
    if out is None:
        with _On(stream):
            out = torch.empty((Bn, H), dtype=kind, device=dev)
    else:
        _check("out", out, (Bn, H), kind, dev, True)
    _run("mccb_scan_step", args, state.data_ptr(), out.data_ptr(), _handle(stream, dev))
    return out


# -- matrix product with its epilogue ----------------------------------------------------------------
class LinearGrads(NamedTuple):
    x: Optional[torch.Tensor]
    weight: Optional[torch.Tensor]
    bias: Optional[torch.Tensor]


def _rows2(name, t):
    """A [..., C] tensor as [R, C] with evenly spaced, contiguous rows, and the rows' spacing."""
    if t.dim() != 2:
        try:
            t = t.view(-1, t.shape[-1])
        except RuntimeError:
            raise ValueError(f"{name}'s rows are not evenly spaced: make it contiguous") from None
    R, C = t.shape
    if C > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return t, t.stride(0) if R > 1 else C


def _linear_args(x, weight, bias, activation):
    if not isinstance(x, torch.Tensor) or x.dim() < 2:
        raise ValueError("x must be a [...,K] tensor of at least two dimensions")
    x2, x_ld = _rows2("x", x)
    code, dev = _data("x", x2, "MK")
    M, K = x2.shape
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be a [N,K] tensor")
    N = weight.shape[0]
    _check("weight", weight, (N, K), x.dtype, dev)
    weight, w_ld = _rows2("weight", weight)
    if bias is not None:
        _check("bias", bias, (N,), x.dtype, dev, True)
    return LinearArgs(M, K, N, code, _activation(activation, (0, 1, 2, 3, 4)), x2.data_ptr(),
                      weight.data_ptr(), _ptr(bias), x_ld, w_ld), (M, K, N, x.dtype, dev)


def linear_forward(x, weight, bias=None, activation=None, residual=None, return_pre=False, out=None,
                   stream=None):
    """out [...,N] = activation(x weight^T + bias) + residual; x [...,K], weight [N,K], bias [N],
    residual [...,N], activation None, "relu", "silu", "gelu" (tanh form) or "softplus". With
    `return_pre` the result is (out, pre), pre = x weight^T + bias as linear_backward needs it."""
    args, (M, K, N, kind, dev) = _linear_args(x, weight, bias, activation)
    shape = (*x.shape[:-1], N)
    res, res_ld = None, 0
    if residual is not None:
        _check("residual", residual, shape, kind, dev)
        res, res_ld = _rows2("residual", residual)
    with _On(stream):
        if out is None:
            out = torch.empty(shape, dtype=kind, device=dev)
        else:
            _check("out", out, shape, kind, dev, True)
        pre = torch.empty(shape, dtype=kind, device=dev) if return_pre else None
        ws, n = _workspace("mccb_linear_forward_get_workspace_size", args, dev)
    _run("mccb_linear_forward", args, _ptr(res), res_ld, out.data_ptr(), _ptr(pre), _ptr(ws), n,
         _handle(stream, dev))
    return (out, pre) if return_pre else out


def linear_backward(gradOut, x, weight, pre=None, activation=None, grad_x=True, grad_weight=True,
                    grad_bias=True, stream=None) -> LinearGrads:
    """Gradients of linear_forward for gradOut [...,N]: of x, weight and bias, as asked for. `pre` is
    linear_forward's (not needed without an activation). The residual's gradient is gradOut."""
    args, (M, K, N, kind, dev) = _linear_args(x, weight, None, activation)
    shape = (*x.shape[:-1], N)
    _check("gradOut", gradOut, shape, kind, dev)
    go, go_ld = _rows2("gradOut", gradOut)
    if pre is not None:
        _check("pre", pre, shape, kind, dev, True)
    with _On(stream):
        g = LinearGrads(torch.empty(x.shape, dtype=kind, device=dev) if grad_x else None,
                        torch.empty((N, K), dtype=kind, device=dev) if grad_weight else None,
                        torch.empty(N, dtype=kind, device=dev) if grad_bias else None)
        ws, n = _workspace("mccb_linear_backward_get_workspace_size", args, dev)
    _run("mccb_linear_backward", args, go.data_ptr(), go_ld, _ptr(pre), _ptr(g.x), _ptr(g.weight),
         _ptr(g.bias), _ptr(ws), n, _handle(stream, dev))
    return g
