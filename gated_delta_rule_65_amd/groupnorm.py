"""Group norm with an activation over channels-last rows (C ABI in ``include/kda_layer.h``), forward and backward: what the
heads' outputs pass on their way to the output projection.

As in the package's other calls, everything is computed in the library's HIP kernels; this module checks tensors,
allocates outputs and workspaces with torch and passes pointers and torch's current stream.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from . import DTYPE, _aligned_grad, _first_order, _ptr, load_library
from .layer import _expect, _float, _launch, _same_device, _token_stride, _wanted, _ws

ACT = {"none": 0, "silu": 1, "sigmoid": 2}


class GroupNormForm(ctypes.Structure):
    """kda_groupnorm_form of the C ABI."""
    _fields_ = [("x_dtype", ctypes.c_int), ("y_dtype", ctypes.c_int), ("act", ctypes.c_int), ("eps", ctypes.c_float)]


def declare(L):
    """Argument types of the entry points."""
    vp, i64, ci, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    form = ctypes.POINTER(GroupNormForm)
    L.kda_groupnorm_fwd.argtypes = [vp, i64, vp, vp, vp, i64, vp, i64, i64, i64, form, vp]
    L.kda_groupnorm_bwd.argtypes = [vp, i64, vp, vp, vp, i64, vp, vp, vp, vp, vp, i64, i64, i64, form, vp, sz, vp]
    L.kda_groupnorm_fwd.restype = L.kda_groupnorm_bwd.restype = ci
    L.kda_groupnorm_bwd_workspace_bytes.argtypes = [i64, i64, i64]
    L.kda_groupnorm_bwd_workspace_bytes.restype = sz


def group_norm_act_workspace_bytes(tokens: int, groups: int, width: int) -> int:
    return int(load_library().kda_groupnorm_bwd_workspace_bytes(tokens, groups, width))


@functools.lru_cache(maxsize=256)
def _form(x_dtype, y_dtype, act, eps):
    return ctypes.pointer(GroupNormForm(DTYPE[x_dtype], DTYPE[y_dtype], ACT[act], eps))


def _rows(t, name):
    """Elements from one token to the next of [..., C]."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU (got {t.device})")
    return t.shape[-1] if t.is_contiguous() else _token_stride(t.unsqueeze(-2), name)


def _inputs(x, groups, weight, bias, gate, act, eps, dtype):
    _float(x, "x")
    size, device = x.shape, x.device
    if len(size) < 1:
        raise ValueError("x must be [..., C]")
    C = size[-1]
    if groups < 1 or C < 1 or C % groups:
        raise ValueError(f"groups must divide the {C} channels (got {groups})")
    if act not in ACT:
        raise ValueError(f"act must be one of {sorted(ACT)} (got {act!r})")
    x_stride, gate_stride = _rows(x, "x"), 0
    if gate is not None:
        _float(gate, "gate")
        if gate.shape != size:
            raise ValueError(f"gate has shape {tuple(gate.shape)}, expected {tuple(size)}")
        if dtype is not None and gate.dtype != dtype:
            raise TypeError(f"gate must have the outputs' type {dtype} (got {gate.dtype})")
        dtype, gate_stride = gate.dtype, _rows(gate, "gate")
        _same_device(device, gate=gate)
    dtype = x.dtype if dtype is None else dtype
    if dtype not in DTYPE:
        raise TypeError(f"dtype must be float32 or bfloat16 (got {dtype})")
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            _expect(t, name, torch.float32, (C,), device)
    args = (_ptr(x), x_stride, _ptr(weight), _ptr(bias), _ptr(gate), gate_stride)
    return args, x.numel() // C, C // groups, dtype, _form(x.dtype, dtype, act, float(eps))


def group_norm_act_fwd(x: torch.Tensor, groups: int, *, weight: Optional[torch.Tensor] = None,
                       bias: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None, act: str = "silu",
                       eps: float = 1e-5, dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """Group norm of each token's channels with an activation, in one pass.

    x [..., C] (bf16 or fp32), the channels of a token contiguous and the tokens at one stride; `groups` groups of adjacent
    channels, normed each: n = (x - mean) / sqrt(var + eps), z = n * weight + bias (fp32 [C], where given).  Returns
    act(z), or z * act(gate) with ``gate`` (x's shape, strided as x may be), contiguous, in the gate's type, or without one
    in ``dtype`` (default: x's).  act: ``"silu"``, ``"sigmoid"`` or ``"none"``.
    """
    args, tokens, width, dtype, form = _inputs(x, groups, weight, bias, gate, act, eps, dtype)
    y = torch.empty_like(x, dtype=dtype, memory_format=torch.contiguous_format)
    _launch(load_library().kda_groupnorm_fwd, x.device, *args, _ptr(y), tokens, groups, width, form)
    return y


def group_norm_act_bwd(x: torch.Tensor, groups: int, dy: torch.Tensor, *, weight: Optional[torch.Tensor] = None,
                       bias: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None, act: str = "silu",
                       eps: float = 1e-5, output_dweights: bool = True, workspace: Optional[torch.Tensor] = None):
    """Gradients of :func:`group_norm_act_fwd` for dL/dy = dy (contiguous, the outputs' type).  Returns dx (contiguous, x's
    type), dweight and dbias (fp32, summed over tokens in a fixed order; None without ``output_dweights``) and dgate
    (contiguous, the gate's type); None for what was not given."""
    _float(dy, "dy")
    args, tokens, width, dtype, form = _inputs(x, groups, weight, bias, gate, act, eps, dy.dtype)
    _expect(dy, "dy", dtype, x.shape, x.device)
    dx = torch.empty_like(x, memory_format=torch.contiguous_format)
    dgate = torch.empty_like(dy) if gate is not None else None
    dw = db = None
    ws, ws_bytes = None, 0
    if output_dweights and (weight is not None or bias is not None):
        dw, db = (torch.empty(groups * width, dtype=torch.float32, device=x.device) for _ in range(2))
        ws, ws_bytes = _ws(group_norm_act_workspace_bytes(tokens, groups, width), workspace, x.device)
    _launch(load_library().kda_groupnorm_bwd, x.device, *args, _ptr(dy), _ptr(dx), _ptr(dgate), _ptr(dw), _ptr(db), tokens,
            groups, width, form, _ptr(ws), ws_bytes)
    return dx, (dw if weight is not None else None), (db if bias is not None else None), dgate


class GroupNormAct(torch.autograd.Function):
    """Autograd wrapper: ``y = GroupNormAct.apply(x, groups, weight, bias, gate, act, eps, dtype)``; weight, bias and gate
    may be None.  It keeps its inputs; gradients of gradients are refused."""

    @staticmethod
    def forward(ctx, x, groups, weight=None, bias=None, gate=None, act="silu", eps=1e-5, dtype=None):
        y = group_norm_act_fwd(x, groups, weight=weight, bias=bias, gate=gate, act=act, eps=eps, dtype=dtype)
        ctx.groups, ctx.y_dtype, ctx.form = groups, y.dtype, {"act": act, "eps": eps}
        ctx.save_for_backward(x, weight, bias, gate)
        return y

    @staticmethod
    @_first_order
    def backward(ctx, dy):
        x, weight, bias, gate = ctx.saved_tensors
        dx, dw, db, dgate = group_norm_act_bwd(x, ctx.groups, _aligned_grad(dy, ctx.y_dtype), weight=weight, bias=bias,
                                               gate=gate, output_dweights=_wanted(ctx, 2) or _wanted(ctx, 3), **ctx.form)
        return dx, None, dw, db, dgate, None, None, None
