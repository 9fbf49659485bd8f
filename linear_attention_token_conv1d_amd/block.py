"""The operators around the mixer in a hybrid block.

As in the package itself, these functions only marshal arguments: torch-level
properties (device, dtype, strides) are checked here, everything else by the
library, and every step of the computation runs in its HIP kernels.  A call's
tensors lie on one GPU; the call runs on torch's current stream of that GPU,
which need not be the current device.
"""
from __future__ import annotations

import ctypes

import torch

from . import BF16, F32, GdnError, _c_void_p, lib

ACT = {"silu": 1, "sigmoid": 2}
ORDER = {"pre": 0, "post": 1}
_DT = {torch.float32: F32, torch.bfloat16: BF16}
_i32, _i64, _f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_float


class NormArgs(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("dtype", _i32), ("weight_dtype", _i32), ("order", _i32),
                ("activation", _i32), ("heads", _i32), ("width", _i32), ("eps", _f32), ("scale", _f32),
                ("weight_offset", _f32), ("tokens", _i64), ("x", _c_void_p), ("weight", _c_void_p),
                ("gate", _c_void_p), ("residual", _c_void_p), ("y", _c_void_p), ("sum", _c_void_p),
                ("x_stride", _i64), ("gate_stride", _i64), ("residual_stride", _i64), ("y_stride", _i64),
                ("sum_stride", _i64)]


class NormBwdArgs(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("dtype", _i32), ("weight_dtype", _i32), ("order", _i32),
                ("activation", _i32), ("heads", _i32), ("width", _i32), ("eps", _f32), ("scale", _f32),
                ("weight_offset", _f32), ("tokens", _i64), ("x", _c_void_p), ("weight", _c_void_p),
                ("gate", _c_void_p), ("dy", _c_void_p), ("d_sum", _c_void_p), ("dx", _c_void_p),
                ("d_residual", _c_void_p), ("dgate", _c_void_p), ("dweight", _c_void_p), ("x_stride", _i64),
                ("gate_stride", _i64), ("dy_stride", _i64), ("d_sum_stride", _i64), ("dx_stride", _i64),
                ("d_residual_stride", _i64), ("dgate_stride", _i64), ("workspace", _c_void_p),
                ("workspace_bytes", ctypes.c_size_t)]


def declare(L):
    """Argument types of this module's entry points in the loaded library."""
    for name, argt in (("gdn_rms_norm", NormArgs), ("gdn_rms_norm_backward", NormBwdArgs)):
        f = getattr(L, name)
        f.argtypes = [ctypes.POINTER(argt), _c_void_p]
        f.restype = ctypes.c_int
    for name, argt in (("gdn_rms_norm_backward_workspace_size", NormBwdArgs),):
        f = getattr(L, name)
        f.argtypes = [ctypes.POINTER(argt)]
        f.restype = ctypes.c_size_t


def _run(name, args, index):
    """Call an entry point on the current stream of GPU `index`."""
    L = lib()
    f = getattr(L, name)
    if index == torch.cuda.current_device():
        status = f(args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            status = f(args, torch._C._cuda_getCurrentRawStream(index))
    if status:
        raise GdnError(f"{name}: {L.gdn_status_string(status).decode()}: {L.gdn_last_error().decode()}")


def _gpu(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise GdnError(f"{name} must be a GPU tensor")
    return t.get_device()


def _tensor(t, name, index, shape, dtype):
    """An optional contiguous tensor of exactly this shape and dtype on GPU `index`: its address."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.get_device() != index:
        raise GdnError(f"{name} must be on the same GPU as the call's other tensors")
    if t.dtype != dtype:
        raise GdnError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise GdnError(f"{name} must be contiguous {list(shape)}, got {list(t.shape)}")
    return t.data_ptr()


def _rows(t, name, index, shape, dtype):
    """An optional [T, H, d] or [T, d] tensor, token stride free: its address and token stride."""
    if t is None:
        return None, 0
    if not isinstance(t, torch.Tensor) or t.get_device() != index:
        raise GdnError(f"{name} must be on the same GPU as the call's other tensors")
    if t.dtype != dtype:
        raise GdnError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise GdnError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    s = t.stride()
    # a stride over one element, or none at all, says nothing about the layout
    if (s[-1] != 1 and shape[-1] > 1) or (len(s) == 3 and s[1] != shape[2] and shape[1] > 1):
        raise GdnError(f"{name} must have contiguous heads inside a token")
    return t.data_ptr(), (s[0] if shape[0] > 1 else t[0].numel() if shape[0] else 0)


def _norm_shape(x):
    index = _gpu(x, "x")
    if x.dtype not in _DT:
        raise GdnError(f"x must be torch.bfloat16 or torch.float32, got {x.dtype}")
    if x.dim() not in (2, 3):
        raise GdnError("x must be [T, D] or [T, H, D]")
    return index, x.shape, (x.shape[1] if x.dim() == 3 else 1), x.shape[-1]


def _norm_how(weight, gate, order, activation):
    if order not in ORDER:
        raise GdnError(f"order must be 'pre' or 'post', got {order!r}")
    if gate is not None and activation not in ACT:
        raise GdnError(f"activation must be 'silu' or 'sigmoid', got {activation!r}")
    if weight is not None and (not isinstance(weight, torch.Tensor) or weight.dtype not in _DT):
        raise GdnError("weight must be a torch.bfloat16 or torch.float32 tensor")
    return ORDER[order], ACT[activation] if gate is not None else 0


def rms_norm(x, weight=None, gate=None, residual=None, order="pre", activation="silu", scale=1.0, eps=1e-6,
             weight_offset=0.0, out=None, sum_out=None):
    """RMS norm over the last dimension of x [T, D] or [T, H, D] (bf16 or fp32,
    token stride free), fused with the residual sum and the output gate.

    order="pre":  h = residual + scale * x; returns (y, h) with a residual, y
    without one, where y = norm(h) * (weight + weight_offset) * act(gate).
    order="post": returns y = residual + scale * norm(x) * (weight + weight_offset) * act(gate).

    weight [D] (bf16 or fp32), gate and residual (like x) are optional;
    activation is "silu" or "sigmoid".  out and sum_out may be given, also as
    the input they replace (in place)."""
    index, shape, heads, width = _norm_shape(x)
    order, act = _norm_how(weight, gate, order, activation)
    dt = x.dtype
    y = torch.empty(shape, dtype=dt, device=x.device) if out is None else out
    sums = residual is not None and order == 0
    if sums and sum_out is None:
        sum_out = torch.empty(shape, dtype=dt, device=x.device)
    if not sums and sum_out is not None:
        raise GdnError("sum_out goes with a residual in the pre order")
    px, sx = _rows(x, "x", index, shape, dt)
    pg, sg = _rows(gate, "gate", index, shape, dt)
    pr, sr = _rows(residual, "residual", index, shape, dt)
    py, sy = _rows(y, "out", index, shape, dt)
    ps, ss = _rows(sum_out, "sum_out", index, shape, dt)
    pw = _tensor(weight, "weight", index, (width,), weight.dtype) if weight is not None else None
    a = NormArgs(ctypes.sizeof(NormArgs), _DT[dt], F32 if weight is None else _DT[weight.dtype], order, act, heads, width,
                 eps, scale, weight_offset, shape[0], px, pw, pg, pr, py, ps, sx, sg, sr, sy, ss)
    _run("gdn_rms_norm", a, index)
    return (y, sum_out) if sums else y


def rms_norm_backward(x, dy, weight=None, gate=None, d_sum=None, residual=False, order="pre", activation="silu",
                      scale=1.0, eps=1e-6, weight_offset=0.0, dx=None, dgate=None, workspace=None):
    """Gradients of rms_norm: returns (dx, dresidual, dweight, dgate).

    x is what was normed: the forward call's x, or the sum h that it returned
    (residual=True, or d_sum, the gradient that reaches h from its other uses,
    say so).  dx is the gradient of the forward call's x; dresidual that of
    the residual (None without one; in the post order it is dy itself and
    None here; with scale 1 it is the same tensor as dx).  dweight is fp32
    [D] (None without a weight), dgate like x (None without a gate)."""
    index, shape, heads, width = _norm_shape(x)
    order, act = _norm_how(weight, gate, order, activation)
    dt, dev = x.dtype, x.device
    residual = residual or d_sum is not None
    if residual and order == 1:
        raise GdnError("residual and d_sum belong to the pre order: in the post order the residual's gradient is dy")
    if order == 0 and not residual and scale != 1.0:
        raise GdnError("the pre order scales x only where it is added to a residual")
    dx = torch.empty(shape, dtype=dt, device=dev) if dx is None else dx
    dres = None
    if residual:
        dres = dx if scale == 1.0 else torch.empty(shape, dtype=dt, device=dev)
    if gate is not None and dgate is None:
        dgate = torch.empty(shape, dtype=dt, device=dev)
    px, sx = _rows(x, "x", index, shape, dt)
    pg, sg = _rows(gate, "gate", index, shape, dt)
    pd, sd = _rows(dy, "dy", index, shape, dt)
    pu, su = _rows(d_sum, "d_sum", index, shape, dt)
    po, so = _rows(dx, "dx", index, shape, dt)
    pr, sr = (None, 0) if dres is dx else _rows(dres, "dresidual", index, shape, dt)
    pz, sz = _rows(dgate, "dgate", index, shape, dt)
    dweight = pw = None
    if weight is not None:
        pw = _tensor(weight, "weight", index, (width,), weight.dtype)
        dweight = torch.empty(width, dtype=torch.float32, device=dev)
    a = NormBwdArgs(ctypes.sizeof(NormBwdArgs), _DT[dt], F32 if weight is None else _DT[weight.dtype], order, act, heads,
                    width, eps, scale, weight_offset, shape[0], px, pw, pg, pd, pu, po, pr, pz,
                    None if dweight is None else dweight.data_ptr(), sx, sg, sd, su, so, sr, sz)
    if dweight is not None:
        workspace = _workspace(workspace, lib().gdn_rms_norm_backward_workspace_size(a), index, dev)
        a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel()
    _run("gdn_rms_norm_backward", a, index)
    return dx, dres, dweight, dgate


def _workspace(given, need, index, dev):
    """The caller's workspace where it is large enough, else a new one."""
    if given is not None:
        if not isinstance(given, torch.Tensor) or given.get_device() != index or given.dtype != torch.uint8:
            raise GdnError("workspace must be a torch.uint8 tensor on the call's GPU")
        if given.numel() >= need and given.is_contiguous():
            return given
    return torch.empty(need, dtype=torch.uint8, device=dev)
