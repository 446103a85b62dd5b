"""Linear attention with a decay for each head (C ABI in ``include/kda_layer.h``): prompts in equal lengths or packed, single
tokens, and the backward pass.

As in the package's other calls, everything is computed in the library's HIP kernels; this module checks tensors,
allocates outputs and workspaces with torch and passes pointers and torch's current stream.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import DTYPE, _aligned_grad, _first_order, _need, _ptr, layer, load_library
from .layer import _expect, _launch, _same_device, _seqs, _wanted, _ws


def declare(L):
    """Argument types of the entry points."""
    vp, i64, ci, sz, f = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
    dims = [ci, ci, ci, f, ci]
    for name, args in {
        "kda_linattn_fwd": [vp] * 7 + [i64, i64] + dims + [vp, sz, vp],
        "kda_linattn_varlen_fwd": [vp] * 5 + [i64, i64] + [vp] * 3 + dims + [vp, sz, vp],
        "kda_linattn_bwd": [vp] * 11 + [i64, i64] + dims + [vp, sz, vp],
        "kda_linattn_varlen_bwd": [vp] * 5 + [i64, i64] + [vp] * 7 + dims + [vp, sz, vp],
        "kda_linattn_step": [vp] * 7 + [i64] + dims + [vp],
    }.items():
        getattr(L, name).argtypes, getattr(L, name).restype = args, ci
    for name in ("kda_linattn_workspace_bytes", "kda_linattn_bwd_workspace_bytes"):
        getattr(L, name).argtypes, getattr(L, name).restype = [i64, i64, ci, ci, ci, ci], sz


def linattn_workspace_bytes(N: int, total: int, H: int, Dk: int, Dv: int, dtype: torch.dtype) -> int:
    return int(load_library().kda_linattn_workspace_bytes(N, total, H, Dk, Dv, DTYPE[dtype]))


def linattn_bwd_workspace_bytes(N: int, total: int, H: int, Dk: int, Dv: int, dtype: torch.dtype) -> int:
    return int(load_library().kda_linattn_bwd_workspace_bytes(N, total, H, Dk, Dv, DTYPE[dtype]))


def _inputs(q, k, v, g, lead):
    """Checks q, k, v and g; returns the leading sizes, H, Dk, Dv."""
    for t, name in ((q, "q"), (v, "v")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
    dtype, size = q.dtype, q.shape
    if len(size) != lead + 2:
        raise ValueError(f"q must be [{'B, T' if lead == 2 else 'B or total'}, H, Dk]")
    if dtype not in DTYPE:
        raise TypeError(f"q, k and v must be float32 or bfloat16 (got {dtype})")
    *front, H, Dk = size
    if v.dim() != lead + 2:
        raise ValueError(f"v has shape {tuple(v.shape)}, expected {(*front, H)} and its own head size")
    Dv, device = v.shape[-1], q.device
    _need(q, "q", dtype)
    _expect(k, "k", dtype, size, device)
    _expect(v, "v", dtype, size if Dv == Dk else (*front, H, Dv), device)
    _expect(g, "g", torch.float32, (H,), device)
    return front, H, Dk, Dv


def _state_like(t, name, shape, device):
    if t is not None:
        _expect(t, name, torch.float32, shape, device)


def _fwd(q, k, v, g, cu, s0, scale, output_final_state, workspace):
    packed = cu is not None
    front, H, Dk, Dv = _inputs(q, k, v, g, 1 if packed else 2)
    N, total = (_seqs(cu), front[0]) if packed else (front[0], front[0] * front[1])
    _same_device(q.device, cu_seqlens=cu)
    _state_like(s0, "s0", (N, H, Dk, Dv), q.device)
    o = torch.empty(v.shape, dtype=q.dtype, device=q.device)
    sf = torch.empty((N, H, Dk, Dv), dtype=torch.float32, device=q.device) if output_final_state else None
    ws, ws_bytes = _ws(linattn_workspace_bytes(N, total, H, Dk, Dv, q.dtype), workspace, q.device)
    tail = (H, Dk, Dv, scale, DTYPE[q.dtype], _ptr(ws), ws_bytes)
    L = load_library()
    if packed:
        _launch(L.kda_linattn_varlen_fwd, q.device, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(cu), N, total, _ptr(s0),
                _ptr(o), _ptr(sf), *tail)
    else:
        _launch(L.kda_linattn_fwd, q.device, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(s0), _ptr(o), _ptr(sf), *front,
                *tail)
    return o, sf


def linattn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, s0: Optional[torch.Tensor] = None, *,
                scale: float = 1.0, output_final_state: bool = True, workspace: Optional[torch.Tensor] = None):
    """Linear attention with a decay for each head: S_t = a S_{t-1} + k_t v_t^T, o_t = scale * S_t^T q_t with
    a = exp(min(g, 0)) of the head.

    q, k: [B, T, H, Dk], v: [B, T, H, Dv] (bf16 or fp32, Dk and Dv 64 or 128); g (fp32): [H], the log of the decay, a
    constant of the layer; s0 (fp32): [B, H, Dk, Dv] or None.  Returns o (v's shape, q's type) and the final state (fp32, or
    None)."""
    return _fwd(q, k, v, g, None, s0, scale, output_final_state, workspace)


def linattn_varlen_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, cu_seqlens: torch.Tensor,
                       s0: Optional[torch.Tensor] = None, *, scale: float = 1.0, output_final_state: bool = True,
                       workspace: Optional[torch.Tensor] = None):
    """:func:`linattn_fwd` over packed sequences: q, k [total, H, Dk], v [total, H, Dv], cu_seqlens int32 [N+1] on the GPU,
    s0 [N, H, Dk, Dv] or None.  Rows behind the last sequence are left unwritten in o."""
    if cu_seqlens is None:
        raise ValueError("cu_seqlens is needed")
    return _fwd(q, k, v, g, cu_seqlens, s0, scale, output_final_state, workspace)


def _bwd(q, k, v, g, cu, d_o, s0, d_sfinal, scale, output_ds0, workspace):
    packed = cu is not None
    front, H, Dk, Dv = _inputs(q, k, v, g, 1 if packed else 2)
    N, total = (_seqs(cu), front[0]) if packed else (front[0], front[0] * front[1])
    _same_device(q.device, cu_seqlens=cu)
    _expect(d_o, "d_o", q.dtype, v.shape, q.device)
    _state_like(s0, "s0", (N, H, Dk, Dv), q.device)
    _state_like(d_sfinal, "d_sfinal", (N, H, Dk, Dv), q.device)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ds0 = torch.empty((N, H, Dk, Dv), dtype=torch.float32, device=q.device) if output_ds0 else None
    ws, ws_bytes = _ws(linattn_bwd_workspace_bytes(N, total, H, Dk, Dv, q.dtype), workspace, q.device)
    tail = (H, Dk, Dv, scale, DTYPE[q.dtype], _ptr(ws), ws_bytes)
    outs = (_ptr(d_o), _ptr(d_sfinal), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ds0))
    L = load_library()
    if packed:
        _launch(L.kda_linattn_varlen_bwd, q.device, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(cu), N, total, _ptr(s0),
                *outs, *tail)
    else:
        _launch(L.kda_linattn_bwd, q.device, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(s0), *outs, *front, *tail)
    return dq, dk, dv, ds0


def linattn_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, d_o: torch.Tensor,
                s0: Optional[torch.Tensor] = None, d_sfinal: Optional[torch.Tensor] = None, *, scale: float = 1.0,
                output_ds0: bool = True, workspace: Optional[torch.Tensor] = None):
    """Gradients of :func:`linattn_fwd` for dL/do = d_o (q's type) and dL/dS_T = d_sfinal (fp32, None = 0).  Returns dq, dk,
    dv (q's type) and ds0 (fp32, or None)."""
    return _bwd(q, k, v, g, None, d_o, s0, d_sfinal, scale, output_ds0, workspace)


def linattn_varlen_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, cu_seqlens: torch.Tensor,
                       d_o: torch.Tensor, s0: Optional[torch.Tensor] = None, d_sfinal: Optional[torch.Tensor] = None, *,
                       scale: float = 1.0, output_ds0: bool = True, workspace: Optional[torch.Tensor] = None):
    """Gradients of :func:`linattn_varlen_fwd`; arguments and results as for :func:`linattn_bwd`.  Rows behind the last
    sequence are left unwritten."""
    if cu_seqlens is None:
        raise ValueError("cu_seqlens is needed")
    return _bwd(q, k, v, g, cu_seqlens, d_o, s0, d_sfinal, scale, output_ds0, workspace)


def linattn_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, state: torch.Tensor, *,
                 scale: float = 1.0, inplace: bool = False) -> Tuple[torch.Tensor, torch.Tensor]:
    """One token per sequence: q, k [B, H, Dk], v [B, H, Dv], state (fp32) [B, H, Dk, Dv].  Returns o [B, H, Dv] (q's type)
    and the new state (``state`` itself when ``inplace``)."""
    (B,), H, Dk, Dv = _inputs(q, k, v, g, 1)
    _expect(state, "state", torch.float32, (B, H, Dk, Dv), q.device)
    o = torch.empty_like(v)
    out = state if inplace else torch.empty_like(state)
    _launch(load_library().kda_linattn_step, q.device, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(state), _ptr(out), _ptr(o),
            B, H, Dk, Dv, scale, DTYPE[q.dtype])
    return o, out


def _constant(ctx, index):
    if ctx.needs_input_grad[index]:
        raise ValueError("g has no gradient here, the decays are constants: pass it detached")


def _state_grad(d_sf):
    return None if d_sf is None else _aligned_grad(d_sf, torch.float32)


class LinearAttention(torch.autograd.Function):
    """Autograd wrapper: ``o, s_final = LinearAttention.apply(q, k, v, g, s0, scale, output_final_state)``; s0 may be None.  Without
    ``output_final_state`` s_final is None, and no state is written forward nor read as its gradient: 64 KB each for a sequence and
    head of 128 channels.  The decays are constants; gradients of gradients are refused."""

    @staticmethod
    def forward(ctx, q, k, v, g, s0=None, scale=1.0, output_final_state=True):
        o, sf = linattn_fwd(q, k, v, g, s0, scale=scale, output_final_state=output_final_state)
        ctx.scale = scale
        ctx.save_for_backward(q, k, v, g, s0)
        return o, sf

    @staticmethod
    @_first_order
    def backward(ctx, d_o, d_sf):
        _constant(ctx, 3)
        q, k, v, g, s0 = ctx.saved_tensors
        wanted = _wanted(ctx, 4)
        dq, dk, dv, ds0 = linattn_bwd(q, k, v, g, _aligned_grad(d_o, q.dtype), s0, _state_grad(d_sf), scale=ctx.scale,
                                      output_ds0=wanted)
        return dq, dk, dv, None, (ds0 if wanted else None), None, None


class VarlenLinearAttention(torch.autograd.Function):
    """:class:`LinearAttention` over packed sequences: ``o, s_final = VarlenLinearAttention.apply(q, k, v, g, cu_seqlens, s0,
    scale, output_final_state)``.  Rows behind the last sequence, where q is longer, are zeros in o and have zero gradients."""

    @staticmethod
    def forward(ctx, q, k, v, g, cu_seqlens, s0=None, scale=1.0, output_final_state=True):
        o, sf = linattn_varlen_fwd(q, k, v, g, cu_seqlens, s0, scale=scale, output_final_state=output_final_state)
        layer._zero_behind(cu_seqlens, o)
        ctx.scale = scale
        ctx.save_for_backward(q, k, v, g, cu_seqlens, s0)
        return o, sf

    @staticmethod
    @_first_order
    def backward(ctx, d_o, d_sf):
        _constant(ctx, 3)
        q, k, v, g, cu, s0 = ctx.saved_tensors
        wanted = _wanted(ctx, 5)
        dq, dk, dv, ds0 = linattn_varlen_bwd(q, k, v, g, cu, _aligned_grad(d_o, q.dtype), s0, _state_grad(d_sf), scale=ctx.scale,
                                             output_ds0=wanted)
        layer._zero_behind(cu, dq, dk)
        layer._zero_behind(cu, dv)
        return dq, dk, dv, None, None, (ds0 if wanted else None), None, None
