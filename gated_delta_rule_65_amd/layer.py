"""The operators around the recurrence (C ABI in ``include/kda_layer.h``): the gated scan over channels, the head
norm of queries and keys with the position rotation, and activation checkpoints in 8 bits.

As in the package's other calls, everything is computed in the library's HIP kernels; this module checks tensors,
allocates outputs and workspaces with torch and passes pointers and torch's current stream.  The autograd functions give
first-order gradients: the gradient of a gradient is refused.
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import NamedTuple, Optional, Tuple

import torch

from . import DTYPE, _aligned_grad, _check, _first_order, _need, _ptr, _stream, chunk_bwd, chunk_fwd, load_library

NORM = {"l2": 0, "rms": 1}


class ScanForm(ctypes.Structure):
    """kda_scan_form of the C ABI."""
    _fields_ = [("x_dtype", ctypes.c_int), ("g_dtype", ctypes.c_int), ("g_logit", ctypes.c_int),
                ("complement", ctypes.c_int)]


class QkNormForm(ctypes.Structure):
    """kda_qknorm_form of the C ABI."""
    _fields_ = [("norm", ctypes.c_int), ("eps", ctypes.c_float), ("rot", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("pos_bytes", ctypes.c_int)]


def declare(L):
    """Argument types of the entry points."""
    vp, i64, ci, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    sf, qf = ctypes.POINTER(ScanForm), ctypes.POINTER(QkNormForm)
    for name, args in {
        "kda_ckpt8_pack": [vp, vp, vp, i64, i64, ci, vp],
        "kda_ckpt8_unpack": [vp, vp, vp, i64, i64, ci, vp],
        "kda_scan_fwd": [vp] * 8 + [i64, i64, i64, sf, vp, sz, vp],
        "kda_scan_varlen_fwd": [vp] * 3 + [i64, i64] + [vp] * 6 + [i64, sf, vp, sz, vp],
        "kda_scan_bwd": [vp] * 11 + [i64, i64, i64, sf, vp, sz, vp],
        "kda_scan_varlen_bwd": [vp] * 3 + [i64, i64] + [vp] * 9 + [i64, sf, vp, sz, vp],
        "kda_scan_zero_behind": [vp, i64, i64, vp, i64, vp, i64, vp],
        "kda_scan_step": [vp] * 5 + [i64, i64, sf, vp],
        "kda_qknorm_fwd": [vp] * 4 + [i64, i64] + [vp] * 10 + [i64, ci, ci, ci, ci, qf, vp],
        "kda_qknorm_bwd": [vp] * 4 + [i64, i64] + [vp] * 10 + [i64, ci, ci, ci, ci, ci, qf, vp, sz, vp],
    }.items():
        getattr(L, name).argtypes, getattr(L, name).restype = args, ci
    for name, args in {"kda_scan_workspace_bytes": [i64] * 3, "kda_scan_carry_bytes": [i64] * 3,
                       "kda_qknorm_bwd_workspace_bytes": [i64, ci, ci, ci]}.items():
        getattr(L, name).argtypes, getattr(L, name).restype = args, sz


def _launch(entry, device, *args):
    """Call an entry point of the library with torch's current stream on `device` as its last argument."""
    index = device.index
    if index == _current_device():
        status = entry(*args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            status = entry(*args, _raw_stream(index))
    if status != 0:
        _check(status)


# The host's share of a call of a few microseconds counts: torch's own short ways to these two, where it has them.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda index: _stream(torch.device("cuda", index)))


def _same_device(device, **tensors):
    index = device.index
    for name, t in tensors.items():
        if t is not None and t.get_device() != index:
            raise ValueError(f"{name} must be on {device} (got {t.device})")


def _float(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in DTYPE:
        raise TypeError(f"{name} must be float32 or bfloat16 (got {t.dtype})")


# ----------------------------------------------------------------- checkpoints in 8 bits

class Packed8(NamedTuple):
    """An activation packed in 8 bits: ``codes`` (uint8, its shape), ``scales`` (uint8, one for each 32 values of the
    last dimension) and the type it came in."""
    codes: torch.Tensor
    scales: torch.Tensor
    dtype: torch.dtype


def _blocks(cols: int) -> int:
    return -(-cols // 32)


def _empty8(shape, dtype, device) -> Packed8:
    return Packed8(torch.empty(shape, dtype=torch.uint8, device=device),
                   torch.empty((*shape[:-1], _blocks(shape[-1])), dtype=torch.uint8, device=device), dtype)


def _need8(p, name: str, shape=None):
    if not isinstance(p, Packed8):
        raise TypeError(f"{name} must be a Packed8")
    _need(p.codes, f"{name}.codes", torch.uint8, shape)
    if p.codes.dim() < 1:
        raise ValueError(f"{name}.codes needs at least one dimension")
    _need(p.scales, f"{name}.scales", torch.uint8, (*p.codes.shape[:-1], _blocks(p.codes.shape[-1])))
    _same_device(p.codes.device, **{f"{name}.scales": p.scales})
    if p.dtype not in DTYPE:
        raise TypeError(f"{name}.dtype must be float32 or bfloat16 (got {p.dtype})")


def ckpt8_pack(x: torch.Tensor) -> Packed8:
    """Pack ``x`` (bf16 or fp32, contiguous) in 8 bits: e4m3 codes with a power-of-two scale for each 32 values of a
    row of the last dimension.  Infinities and NaN become NaN."""
    _float(x, "x")
    _need(x, "x")
    if x.dim() < 1:
        raise ValueError("x needs at least one dimension")
    cols = x.shape[-1]
    out = _empty8(x.shape, x.dtype, x.device)
    _launch(load_library().kda_ckpt8_pack, x.device, _ptr(x), _ptr(out.codes), _ptr(out.scales), x.numel() // cols if
            cols else 0, cols, DTYPE[x.dtype])
    return out


def ckpt8_unpack(packed: Packed8, dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """The values that a packed activation stands for, in ``dtype`` (default: the type it came in); exact in both."""
    _need8(packed, "packed")
    dtype = packed.dtype if dtype is None else dtype
    if dtype not in DTYPE:
        raise TypeError(f"dtype must be float32 or bfloat16 (got {dtype})")
    cols, device = packed.codes.shape[-1], packed.codes.device
    x = torch.empty(packed.codes.shape, dtype=dtype, device=device)
    _launch(load_library().kda_ckpt8_unpack, device, _ptr(packed.codes), _ptr(packed.scales), _ptr(x), x.numel() //
            cols if cols else 0, cols, DTYPE[dtype])
    return x


# ----------------------------------------------------------------- gated scan over channels

def scan_workspace_bytes(N: int, total: int, D: int) -> int:
    return int(load_library().kda_scan_workspace_bytes(N, total, D))


def scan_carry_bytes(N: int, total: int, D: int) -> int:
    return int(load_library().kda_scan_carry_bytes(N, total, D))


@functools.lru_cache(maxsize=None)
def _form(x_dtype, g_dtype, g_logit, complement):
    return ctypes.pointer(ScanForm(DTYPE[x_dtype], DTYPE[g_dtype], int(bool(g_logit)), int(bool(complement))))


@functools.lru_cache(maxsize=256)
def _qk_form(norm, eps, rot, interleaved, pos_bytes):
    return ctypes.pointer(QkNormForm(NORM[norm], eps, rot, int(bool(interleaved)), pos_bytes))


def _ws(need: int, workspace: Optional[torch.Tensor], device) -> Tuple[Optional[torch.Tensor], int]:
    if need == 0:
        return None, 0
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    else:
        _need(workspace, "workspace")
        _same_device(device, workspace=workspace)
    return workspace, workspace.numel() * workspace.element_size()


def _seqs(cu_seqlens: torch.Tensor) -> int:
    _need(cu_seqlens, "cu_seqlens", torch.int32)
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be one-dimensional with at least one entry")
    return cu_seqlens.numel() - 1


def _scan_fwd(x, g, cu, h0, g_logit, complement, output_final_state, save, workspace):
    lead = 1 if cu is not None else 2
    if not isinstance(x, torch.Tensor) or x.dim() <= lead:
        raise ValueError("x must be [total, channels...]" if cu is not None else "x must be [B, T, channels...]")
    _float(x, "x")
    _float(g, "g")
    _need(x, "x")
    _need(g, "g", None, x.shape)
    chans = tuple(x.shape[lead:])
    D, N = math.prod(chans), _seqs(cu) if cu is not None else x.shape[0]
    total = x.shape[0] if cu is not None else x.shape[0] * x.shape[1]
    if h0 is not None:
        _need(h0, "h0", torch.float32, (N, *chans))
    _same_device(x.device, g=g, h0=h0, cu_seqlens=cu)
    if save not in (None, "carry", "ckpt8"):
        raise ValueError(f"save must be None, 'carry' or 'ckpt8' (got {save!r})")
    y = torch.empty_like(x)
    hf = torch.empty((N, *chans), dtype=torch.float32, device=x.device) if output_final_state else None
    carry = u = saved = None
    if save == "carry":
        saved = carry = torch.empty(scan_carry_bytes(N, total, D) // 4, dtype=torch.float32, device=x.device)
    elif save == "ckpt8":
        saved = u = _empty8((total, D), x.dtype, x.device)
    ws, ws_bytes = _ws(scan_workspace_bytes(N, total, D), workspace, x.device)
    u_ptrs = (_ptr(u.codes), _ptr(u.scales)) if u is not None else (None, None)
    form = _form(x.dtype, g.dtype, bool(g_logit), bool(complement))
    L = load_library()
    if cu is None:
        _launch(L.kda_scan_fwd, x.device, _ptr(x), _ptr(g), _ptr(h0), _ptr(y), _ptr(hf), _ptr(carry), *u_ptrs,
                x.shape[0], x.shape[1], D, form, _ptr(ws), ws_bytes)
    else:
        _launch(L.kda_scan_varlen_fwd, x.device, _ptr(x), _ptr(g), _ptr(cu), N, total, _ptr(h0), _ptr(y), _ptr(hf),
                _ptr(carry), *u_ptrs, D, form, _ptr(ws), ws_bytes)
    return y, hf, saved


def scan_fwd(x: torch.Tensor, g: torch.Tensor, h0: Optional[torch.Tensor] = None, *, g_logit: bool = False,
             complement: bool = False, output_final_state: bool = True, save: Optional[str] = None,
             workspace: Optional[torch.Tensor] = None):
    """Gated scan over channels: h_t = a_t h_{t-1} + w_t x_t per sequence and channel, y_t = h_t.

    x, g: [B, T, channels...] (bf16 or fp32, each its own); a_t = exp(clamp(g, -5, 0)), or with ``g_logit``
    exp(clamp(-softplus(g), -5, 0)); w_t = 1, or 1 - a_t with ``complement``.  h0 (fp32): [B, channels...] or None.
    Returns y (x's type), the final state (fp32, or None) and what :func:`scan_bwd` needs beside g:
    ``save="carry"``, the state at every 64th token (with x it gives the exact gradients), or ``save="ckpt8"``, the
    factor of the gates' gradient in 8 bits (x is not needed then); else None.
    """
    return _scan_fwd(x, g, None, h0, g_logit, complement, output_final_state, save, workspace)


def scan_varlen_fwd(x: torch.Tensor, g: torch.Tensor, cu_seqlens: torch.Tensor, h0: Optional[torch.Tensor] = None, *,
                    g_logit: bool = False, complement: bool = False, output_final_state: bool = True,
                    save: Optional[str] = None, workspace: Optional[torch.Tensor] = None):
    """:func:`scan_fwd` over packed sequences: x, g [total, channels...], cu_seqlens int32 [N+1] on the GPU, h0
    [N, channels...] or None.  Rows behind the last sequence are left unwritten in y."""
    return _scan_fwd(x, g, cu_seqlens, h0, g_logit, complement, output_final_state, save, workspace)


def _scan_bwd(g, dy, cu, saved, x, h0, dh_final, g_logit, complement, workspace):
    lead = 1 if cu is not None else 2
    if not isinstance(dy, torch.Tensor) or dy.dim() <= lead:
        raise ValueError("dy must be [total, channels...]" if cu is not None else "dy must be [B, T, channels...]")
    _float(g, "g")
    _float(dy, "dy")
    _need(dy, "dy")
    _need(g, "g", None, dy.shape)
    chans = tuple(dy.shape[lead:])
    D, N = math.prod(chans), _seqs(cu) if cu is not None else dy.shape[0]
    total = dy.shape[0] if cu is not None else dy.shape[0] * dy.shape[1]
    carry = codes = scales = None
    if isinstance(saved, Packed8):
        _need8(saved, "saved", (total, D))
        codes, scales = saved.codes, saved.scales
        x = h0 = None
    else:
        if x is None:
            raise ValueError("x is needed with the carry that save='carry' gave")
        _need(x, "x", dy.dtype, dy.shape)
        _need(saved, "saved", torch.float32, (scan_carry_bytes(N, total, D) // 4,))
        carry = saved
        if h0 is not None:
            _need(h0, "h0", torch.float32, (N, *chans))
    if dh_final is not None:
        _need(dh_final, "dh_final", torch.float32, (N, *chans))
    _same_device(dy.device, g=g, cu_seqlens=cu, x=x, saved=carry if codes is None else codes, h0=h0, dh_final=dh_final)
    dx, dg = torch.empty_like(dy), torch.empty_like(g)
    dh0 = torch.empty((N, *chans), dtype=torch.float32, device=dy.device)
    ws, ws_bytes = _ws(scan_workspace_bytes(N, total, D), workspace, dy.device)
    form = _form(dy.dtype, g.dtype, bool(g_logit), bool(complement))
    L = load_library()
    if cu is None:
        _launch(L.kda_scan_bwd, dy.device, _ptr(x), _ptr(g), _ptr(h0), _ptr(carry), _ptr(codes), _ptr(scales),
                _ptr(dy), _ptr(dh_final), _ptr(dx), _ptr(dg), _ptr(dh0), dy.shape[0], dy.shape[1], D, form, _ptr(ws),
                ws_bytes)
    else:
        _launch(L.kda_scan_varlen_bwd, dy.device, _ptr(x), _ptr(g), _ptr(cu), N, total, _ptr(h0), _ptr(carry),
                _ptr(codes), _ptr(scales), _ptr(dy), _ptr(dh_final), _ptr(dx), _ptr(dg), _ptr(dh0), D, form, _ptr(ws),
                ws_bytes)
    return dx, dg, dh0


def scan_bwd(g: torch.Tensor, dy: torch.Tensor, saved, *, x: Optional[torch.Tensor] = None,
             h0: Optional[torch.Tensor] = None, dh_final: Optional[torch.Tensor] = None, g_logit: bool = False,
             complement: bool = False, workspace: Optional[torch.Tensor] = None):
    """Gradients of :func:`scan_fwd` for dL/dy = dy (x's type) and dL/dh_T = dh_final (fp32, None = 0).

    ``saved`` is what the forward call returned: its carry, with the same x and h0, or its packed checkpoint (x and h0
    are not read then).  Returns dx (x's type), dg (g's type, with respect to g before the clamp) and dh0 (fp32)."""
    return _scan_bwd(g, dy, None, saved, x, h0, dh_final, g_logit, complement, workspace)


def scan_varlen_bwd(g: torch.Tensor, cu_seqlens: torch.Tensor, dy: torch.Tensor, saved, *,
                    x: Optional[torch.Tensor] = None, h0: Optional[torch.Tensor] = None,
                    dh_final: Optional[torch.Tensor] = None, g_logit: bool = False, complement: bool = False,
                    workspace: Optional[torch.Tensor] = None):
    """Gradients of :func:`scan_varlen_fwd`; arguments and results as for :func:`scan_bwd`."""
    return _scan_bwd(g, dy, cu_seqlens, saved, x, h0, dh_final, g_logit, complement, workspace)


def scan_step(x: torch.Tensor, g: torch.Tensor, state: torch.Tensor, *, inplace: bool = False, g_logit: bool = False,
              complement: bool = False) -> Tuple[torch.Tensor, torch.Tensor]:
    """One token per sequence: x, g [B, channels...], state (fp32) of the same shape.  Returns y (x's type) and
    the new state (``state`` itself when ``inplace``)."""
    if not isinstance(x, torch.Tensor) or x.dim() < 2:
        raise ValueError("x must be [B, channels...]")
    _float(x, "x")
    _float(g, "g")
    _need(x, "x")
    _need(g, "g", None, x.shape)
    _need(state, "state", torch.float32, x.shape)
    _same_device(x.device, g=g, state=state)
    y = torch.empty_like(x)
    out = state if inplace else torch.empty_like(state)
    _launch(load_library().kda_scan_step, x.device, _ptr(x), _ptr(g), _ptr(state), _ptr(out), _ptr(y), x.shape[0],
            math.prod(x.shape[1:]), _form(x.dtype, g.dtype, bool(g_logit), bool(complement)))
    return y, out


class GatedScan(torch.autograd.Function):
    """Autograd wrapper: ``y, h_final = GatedScan.apply(x, g, h0, g_logit, complement, ckpt8)``; h0 may be None.
    With ``ckpt8`` it keeps g and one byte per value for the backward pass, else g, x and the state at every 64th
    token."""

    @staticmethod
    def forward(ctx, x, g, h0=None, g_logit=False, complement=False, ckpt8=False):
        y, hf, saved = scan_fwd(x, g, h0, g_logit=g_logit, complement=complement, save="ckpt8" if ckpt8 else "carry")
        _keep_scan(ctx, x, g, h0, saved, g_logit, complement, ckpt8)
        return y, hf

    @staticmethod
    @_first_order
    def backward(ctx, dy, dh_final):
        g, saved, x, h0, _, form = _kept_scan(ctx)
        dx, dg, dh0 = scan_bwd(g, _aligned_grad(dy, ctx.x_dtype), saved, x=x, h0=h0,
                               dh_final=_aligned_grad(dh_final, torch.float32), **form)
        return dx, dg, (dh0 if ctx.has_h0 else None), None, None, None


class VarlenGatedScan(torch.autograd.Function):
    """:class:`GatedScan` over packed sequences: ``y, h_final = VarlenGatedScan.apply(x, g, cu_seqlens, h0, g_logit,
    complement, ckpt8)``.  Rows behind the last sequence, where x is longer, are zeros in y and have zero gradients."""

    @staticmethod
    def forward(ctx, x, g, cu_seqlens, h0=None, g_logit=False, complement=False, ckpt8=False):
        y, hf, saved = scan_varlen_fwd(x, g, cu_seqlens, h0, g_logit=g_logit, complement=complement,
                                       save="ckpt8" if ckpt8 else "carry")
        _zero_behind(cu_seqlens, y)
        _keep_scan(ctx, x, g, h0, saved, g_logit, complement, ckpt8, cu_seqlens)
        return y, hf

    @staticmethod
    @_first_order
    def backward(ctx, dy, dh_final):
        g, saved, x, h0, cu, form = _kept_scan(ctx)
        dx, dg, dh0 = scan_varlen_bwd(g, cu, _aligned_grad(dy, ctx.x_dtype), saved, x=x, h0=h0,
                                      dh_final=_aligned_grad(dh_final, torch.float32), **form)
        _zero_behind(cu, dx, dg)
        return dx, dg, None, (dh0 if ctx.has_h0 else None), None, None, None


def _zero_behind(cu, a, b=None):
    """Zeros for the rows of a and b [total, channels...] that the calls over packed sequences leave unwritten."""
    total, rows = a.shape[0], [0 if t is None else math.prod(t.shape[1:]) * t.element_size() for t in (a, b)]
    _launch(load_library().kda_scan_zero_behind, a.device, _ptr(cu), cu.numel() - 1, total, _ptr(a), rows[0], _ptr(b), rows[1])


def _keep_scan(ctx, x, g, h0, saved, g_logit, complement, ckpt8, cu=None):
    ctx.x_dtype, ctx.has_h0, ctx.ckpt8 = x.dtype, h0 is not None, ckpt8
    ctx.form = {"g_logit": g_logit, "complement": complement}
    ctx.save_for_backward(cu, g, *((saved.codes, saved.scales) if ckpt8 else (saved, x, h0)))


def _kept_scan(ctx):
    if ctx.ckpt8:
        cu, g, codes, scales = ctx.saved_tensors
        return g, Packed8(codes, scales, ctx.x_dtype), None, None, cu, ctx.form
    cu, g, carry, x, h0 = ctx.saved_tensors
    return g, carry, x, h0, cu, ctx.form


# ----------------------------------------------------------------- head norm with rotation

def qk_norm_rope_workspace_bytes(tokens: int, Hq: int, Hk: int, D: int) -> int:
    return int(load_library().kda_qknorm_bwd_workspace_bytes(tokens, Hq, Hk, D))


def _token_stride(t: torch.Tensor, name: str) -> int:
    """Elements from one token to the next of [..., H, D] whose heads are contiguous and whose leading dimensions lie
    behind one another at one stride."""
    H, D = t.shape[-2:]
    if t.is_contiguous() or t.numel() == 0:
        return H * D
    if t.stride(-1) != 1 or (H > 1 and t.stride(-2) != D):
        raise ValueError(f"the heads of a token of {name} must be contiguous")
    stride = expect = None
    for size, step in zip(reversed(t.shape[:-2]), reversed(t.stride()[:-2])):
        if size == 1:
            continue
        if stride is None:
            stride = step
        elif step != expect:
            raise ValueError(f"the tokens of {name} must lie at one stride")
        expect = step * size
    return H * D if stride is None else stride


def _qk_side(t, name):
    if isinstance(t, Packed8):
        _need8(t, name)
        if t.codes.dim() < 2:
            raise ValueError(f"{name} must be [..., H, D]")
        return t.codes, t.scales, math.prod(t.codes.shape[-2:]), t.dtype
    _float(t, name)
    if t.dim() < 2:
        raise ValueError(f"{name} must be [..., H, D]")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU (got {t.device})")
    return t, None, _token_stride(t, name), t.dtype


def _qk_inputs(q, k, weight_q, weight_k, pos, freqs, norm, eps, interleaved):
    if isinstance(q, Packed8) != isinstance(k, Packed8):
        raise TypeError("q and k must both be packed, or neither")
    qt, qs, q_stride, q_dtype = _qk_side(q, "q")
    kt, ks, k_stride, k_dtype = _qk_side(k, "k")
    if q_dtype != k_dtype:
        raise TypeError(f"q and k must have one type (got {q_dtype} and {k_dtype})")
    lead, D = tuple(qt.shape[:-2]), qt.shape[-1]
    if tuple(kt.shape[:-2]) != lead or kt.shape[-1] != D:
        raise ValueError(f"k has shape {tuple(kt.shape)}, expected {lead} tokens of heads of {D}")
    if weight_q is not None:
        _need(weight_q, "weight_q", torch.float32, (D,))
    if weight_k is not None:
        _need(weight_k, "weight_k", torch.float32, (D,))
    if (pos is None) != (freqs is None):
        raise ValueError("pos and freqs must both be given, or neither")
    rot, pos_bytes = 0, 0
    if pos is not None:
        if not isinstance(pos, torch.Tensor) or pos.dtype not in (torch.int32, torch.int64):
            raise TypeError("pos must be an int32 or int64 tensor")
        _need(pos, "pos", None, lead)
        _need(freqs, "freqs", torch.float64)
        if freqs.dim() != 1:
            raise ValueError("freqs must be one-dimensional, a frequency for each pair")
        rot, pos_bytes = 2 * freqs.numel(), pos.element_size()
    if norm not in NORM:
        raise ValueError(f"norm must be one of {sorted(NORM)} (got {norm!r})")
    _same_device(qt.device, q_scales=qs, k=kt, k_scales=ks, weight_q=weight_q, weight_k=weight_k, pos=pos, freqs=freqs)
    form = _qk_form(norm, float(eps), rot, bool(interleaved), pos_bytes)
    args = (_ptr(qt), _ptr(kt), _ptr(qs), _ptr(ks), q_stride, k_stride, _ptr(weight_q), _ptr(weight_k), _ptr(pos),
            _ptr(freqs))
    return args, math.prod(lead), qt.shape[-2], kt.shape[-2], D, q_dtype, qt.device, form


def qk_norm_rope_fwd(q, k, *, weight_q: Optional[torch.Tensor] = None, weight_k: Optional[torch.Tensor] = None,
                     pos: Optional[torch.Tensor] = None, freqs: Optional[torch.Tensor] = None, norm: str = "l2",
                     eps: float = 0.0, interleaved: bool = False, ckpt8: bool = False):
    """Norm of queries and keys per head and their position rotation, in one pass.

    q [..., Hq, D], k [..., Hk, D] (bf16 or fp32, D 64 or 128), the heads of a token contiguous and the tokens at one
    stride, so that they may be columns of a wider projection; or both :class:`Packed8`.  norm ``"l2"``: x / sqrt(|x|^2
    + eps); ``"rms"``: x / sqrt(mean x^2 + eps); then times weight_q, weight_k (fp32 [D]) where given.  pos
    (int32 or int64 [...]) and freqs (fp64 [R], radians per position) turn the first 2R channels (a multiple of 16):
    pairs (i, i + R), or (2i, 2i + 1) with ``interleaved``.  Returns q, k (contiguous, the inputs' type) and with
    ``ckpt8`` the raw q and k packed in 8 bits (a pair) for the backward pass, else None.
    """
    args, tokens, Hq, Hk, D, dtype, device, form = _qk_inputs(q, k, weight_q, weight_k, pos, freqs, norm, eps,
                                                              interleaved)
    qt, kt = (q.codes, k.codes) if isinstance(q, Packed8) else (q, k)
    q_out = torch.empty(qt.shape, dtype=dtype, device=device)
    k_out = torch.empty(kt.shape, dtype=dtype, device=device)
    saved, ptrs = None, (None,) * 4
    if ckpt8:
        if isinstance(q, Packed8):
            raise ValueError("q and k are packed already")
        saved = (_empty8(q.shape, dtype, device), _empty8(k.shape, dtype, device))
        ptrs = tuple(_ptr(t) for p in saved for t in p[:2])
    _launch(load_library().kda_qknorm_fwd, device, *args, _ptr(q_out), _ptr(k_out), *ptrs, tokens, Hq, Hk, D,
            DTYPE[dtype], form)
    return q_out, k_out, saved


def qk_norm_rope_bwd(q, k, d_q: torch.Tensor, d_k: torch.Tensor, *, weight_q: Optional[torch.Tensor] = None,
                     weight_k: Optional[torch.Tensor] = None, pos: Optional[torch.Tensor] = None,
                     freqs: Optional[torch.Tensor] = None, norm: str = "l2", eps: float = 0.0,
                     interleaved: bool = False, workspace: Optional[torch.Tensor] = None):
    """Gradients of :func:`qk_norm_rope_fwd` for the gradients d_q, d_k of its outputs (contiguous, bf16 or fp32, both
    the same); q and k as given to it, or packed.  Returns dq, dk (contiguous, q's type) and the gradients of
    weight_q and weight_k (fp32, summed over tokens and heads in a fixed order; None where there is no weight)."""
    args, tokens, Hq, Hk, D, dtype, device, form = _qk_inputs(q, k, weight_q, weight_k, pos, freqs, norm, eps,
                                                              interleaved)
    qt, kt = (q.codes, k.codes) if isinstance(q, Packed8) else (q, k)
    _float(d_q, "d_q")
    _need(d_q, "d_q", None, qt.shape)
    _need(d_k, "d_k", d_q.dtype, kt.shape)
    _same_device(device, d_q=d_q, d_k=d_k)
    dq, dk = torch.empty(qt.shape, dtype=dtype, device=device), torch.empty(kt.shape, dtype=dtype, device=device)
    dwq = dwk = None
    ws, ws_bytes = None, 0
    if weight_q is not None or weight_k is not None:
        dwq, dwk = (torch.empty(D, dtype=torch.float32, device=device) for _ in range(2))
        ws, ws_bytes = _ws(qk_norm_rope_workspace_bytes(tokens, Hq, Hk, D), workspace, device)
    _launch(load_library().kda_qknorm_bwd, device, *args, _ptr(d_q), _ptr(d_k), _ptr(dq), _ptr(dk), _ptr(dwq),
            _ptr(dwk), tokens, Hq, Hk, D, DTYPE[dtype], DTYPE[d_q.dtype], form, _ptr(ws), ws_bytes)
    return dq, dk, (dwq if weight_q is not None else None), (dwk if weight_k is not None else None)


class NormChunkKDA(torch.autograd.Function):
    """The recurrence behind the head norm and rotation, with gradients for the raw queries and keys:

        ``o, s_final = NormChunkKDA.apply(q, k, v, g, beta, s0, weight_q, weight_k, pos, freqs, norm, eps,
        interleaved, ckpt8)``

    q, k, v, g, beta, s0 as for :func:`chunk_fwd` (q and k raw, possibly columns of a projection), the rest as for
    :func:`qk_norm_rope_fwd`.  The normed q and k are not kept: the backward pass makes them again.  With ``ckpt8`` it
    keeps the raw q, k and v in 8 bits (3 bytes per channel instead of 6 in bf16) and the gradients are those at the
    values these stand for.  Positions and frequencies are constants."""

    @staticmethod
    def forward(ctx, q, k, v, g, beta, s0=None, weight_q=None, weight_k=None, pos=None, freqs=None, norm="l2",
                eps=0.0, interleaved=False, ckpt8=False):
        ctx.form = {"norm": norm, "eps": eps, "interleaved": interleaved}
        qn, kn, raw = qk_norm_rope_fwd(q, k, weight_q=weight_q, weight_k=weight_k, pos=pos, freqs=freqs, ckpt8=ckpt8,
                                       **ctx.form)
        o, sf = chunk_fwd(qn, kn, v, g, beta, s0)
        ctx.dtype, ctx.ckpt8 = q.dtype, ckpt8
        kept = [t for p in (*raw, ckpt8_pack(v)) for t in p[:2]] if ckpt8 else [q, k, v]
        ctx.save_for_backward(g, beta, s0, weight_q, weight_k, pos, freqs, *kept)
        return o, sf

    @staticmethod
    @_first_order
    def backward(ctx, d_o, d_sf):
        g, beta, s0, weight_q, weight_k, pos, freqs, *kept = ctx.saved_tensors
        if any(ctx.needs_input_grad[9:10]):
            raise ValueError("freqs have no gradient here: pass them detached")
        if ctx.ckpt8:
            q, k, v = (Packed8(kept[2 * i], kept[2 * i + 1], ctx.dtype) for i in range(3))
            v = ckpt8_unpack(v)
        else:
            q, k, v = kept
        form = {"weight_q": weight_q, "weight_k": weight_k, "pos": pos, "freqs": freqs, **ctx.form}
        qn, kn, _ = qk_norm_rope_fwd(q, k, **form)
        # gates of 16 bits stand for their values: 32 bits hold them
        dqn, dkn, dv, dg, dbeta, ds0 = chunk_bwd(qn, kn, v, g.float(), beta.float(), _aligned_grad(d_o, torch.float32),
                                                 s0, _aligned_grad(d_sf, torch.float32))
        dq, dk, dwq, dwk = qk_norm_rope_bwd(q, k, dqn, dkn, **form)
        return (dq, dk, dv.to(ctx.dtype), dg.to(g.dtype), dbeta.to(beta.dtype), ds0 if s0 is not None else None, dwq, dwk,
                None, None, None, None, None, None)
