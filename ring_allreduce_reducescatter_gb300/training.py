"""The operators of a training step around its products: layer norm, the linear
cross entropy, and the orthogonalised update.

The binding of the ``ring_layer_norm*``, ``ring_linear_cross_entropy*`` and
``ring_orthogonalize`` entry points of ``include/ringred.h`` (which defines
them).  As elsewhere in the package only arguments are marshalled here; outputs
and workspaces that are not given are torch tensors allocated on the stream of
the call.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from .mx4 import _current, _dtype, _failed, _matrix, _on, _output

_F32 = torch.float32


def bind(L) -> None:
    """Argument types of the entry points, called once when the library loads."""
    sz, i, vp, f64 = ctypes.c_size_t, ctypes.c_int, ctypes.c_void_p, ctypes.c_double
    L.ring_layer_norm_workspace.argtypes, L.ring_layer_norm_workspace.restype = [sz, sz], sz
    L.ring_layer_norm.argtypes = [vp, sz, vp, vp, i, f64, vp, sz, vp, vp, sz, sz, i, vp]
    L.ring_layer_norm_backward.argtypes = [vp, sz, vp, sz, vp, i, vp, vp, vp, sz, vp, vp, sz, sz, i, vp, sz, vp]
    for f in ("ring_layer_norm", "ring_layer_norm_backward"):
        getattr(L, f).restype = i


_L = None


def _lib():
    global _L
    if _L is None:
        from . import lib

        _L = lib()
    return _L


def _recorded(*ts) -> bool:
    """Whether a gradient of one of these is being recorded."""
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in ts)


def _rows(t, name: str):
    """(rows, cols, row stride) of a tensor whose last axis is the row: any
    contiguous tensor, or a two-dimensional one with neighbouring columns."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name}: needs a CUDA tensor")
    if t.dim() == 2:
        return _matrix(t, name)
    if t.dim() == 0 or not t.is_contiguous():
        raise ValueError(f"{name}: needs a contiguous tensor of one dimension or more, or a two-dimensional one "
                         "with neighbouring columns")
    cols = t.shape[-1]
    return (t.numel() // cols if cols else 0), cols, cols


# ------------------------------------------------------------------ layer norm


def _weights(x, cols, dtype, **named):
    """The C code of the weights' one dtype (x's where there are none)."""
    wtype = None
    for name, t in named.items():
        if t is None:
            continue
        if not isinstance(t, torch.Tensor) or tuple(t.shape) != (cols,) or not t.is_contiguous() or t.device != x.device:
            raise ValueError(f"{name}: needs a contiguous tensor of {cols} elements on {x.device}")
        if t.dtype not in (x.dtype, _F32) or (wtype is not None and t.dtype != wtype):
            raise ValueError(f"{name}: {t.dtype}; the weights have one dtype, x's ({x.dtype}) or float32")
        wtype = t.dtype
    return dtype if wtype is None else _dtype(wtype)


def _at(t):
    return None if t is None else t.data_ptr()


def layer_norm_forward(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                       eps: float = 1e-5, out: Optional[torch.Tensor] = None,
                       stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(y, mean, rstd): layer norm over x's last axis, and each row's mean and
    1 / sqrt(variance + eps) in float32, as layer_norm_backward takes them.
    Records no gradient (layer_norm does)."""
    if stream is not None:
        return _on(stream, layer_norm_forward, x, weight, bias, eps, out)
    if _recorded(x, weight, bias):
        raise ValueError("a gradient is being recorded, and would be lost: layer_norm records it")
    return _norm(x, weight, bias, eps, out, True)


def _norm(x, weight, bias, eps, out, stats):
    rows, cols, ld = _rows(x, "x")
    code, device, handle = _dtype(x.dtype), x.device, _current(x.device)
    wcode = _weights(x, cols, code, weight=weight, bias=bias)
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=device)
        ld_out = cols
    else:
        _, _, ld_out = _rows(out, "out")
        if out.shape != x.shape or out.dtype != x.dtype or out.device != device:
            raise ValueError("x and out must have one shape, dtype and device")
    mean = rstd = None
    if stats:
        both = torch.empty((2,) + tuple(x.shape[:-1]), dtype=_F32, device=device)
        mean, rstd = both[0], both[1]
    status = (_L or _lib()).ring_layer_norm(x.data_ptr(), ld, _at(weight), _at(bias), wcode, eps, out.data_ptr(), ld_out,
                                            _at(mean), _at(rstd), rows, cols, code, handle)
    if status:
        _failed(status, "ring_layer_norm")
    return out, mean, rstd


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        weight: Optional[torch.Tensor] = None, want_dx: bool = True, want_dweight: bool = True,
                        want_dbias: bool = True, wdtype: Optional[torch.dtype] = None, stream=None):
    """(dx, dweight, dbias) of layer norm, None for what is not wanted.  dweight
    and dbias have the weight's dtype, without one wdtype (x's if None)."""
    if stream is not None:
        return _on(stream, layer_norm_backward, dy, x, mean, rstd, weight, want_dx, want_dweight, want_dbias, wdtype)
    rows, cols, ld_x = _rows(x, "x")
    r, c, ld_dy = _rows(dy, "dy")
    device = x.device
    if dy.shape != x.shape or dy.dtype != x.dtype or dy.device != device:
        raise ValueError("x and dy must have one shape, dtype and device")
    for name, t in (("mean", mean), ("rstd", rstd)):
        if (not isinstance(t, torch.Tensor) or t.dtype != _F32 or t.shape != x.shape[:-1] or t.device != device
                or not t.is_contiguous()):
            raise ValueError(f"{name}: needs a contiguous float32 tensor of shape {tuple(x.shape[:-1])} on {device}")
    code, handle = _dtype(x.dtype), _current(device)
    wcode = _weights(x, cols, code, weight=weight)
    wtype = weight.dtype if weight is not None else x.dtype if wdtype is None else wdtype
    if wtype not in (x.dtype, _F32):
        raise ValueError(f"wdtype {wtype}: x's dtype ({x.dtype}) or float32 is wanted")
    wcode = _dtype(wtype)
    dx = torch.empty(x.shape, dtype=x.dtype, device=device) if want_dx else None
    dweight = torch.empty(cols, dtype=wtype, device=device) if want_dweight else None
    dbias = torch.empty(cols, dtype=wtype, device=device) if want_dbias else None
    L = _L or _lib()
    need = L.ring_layer_norm_workspace(rows, cols) if want_dweight or want_dbias else 0
    space = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    status = L.ring_layer_norm_backward(dy.data_ptr(), ld_dy, x.data_ptr(), ld_x, _at(weight), wcode, mean.data_ptr(),
                                        rstd.data_ptr(), _at(dx), cols, _at(dweight), _at(dbias), rows, cols, code,
                                        _at(space), need, handle)
    if status:
        _failed(status, "ring_layer_norm_backward")
    return dx, dweight, dbias


class _Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = _norm(x, weight, bias, eps, None, True)
        ctx.save_for_backward(x, mean, rstd, weight)
        ctx.wdtype = bias.dtype if bias is not None else None
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, mean, rstd, weight = ctx.saved_tensors
        need = ctx.needs_input_grad
        if dy.dim() != 2 or dy.stride(1) != 1 or dy.stride(0) < dy.shape[1]:
            dy = dy.contiguous()
        return layer_norm_backward(dy, x, mean, rstd, weight, need[0], need[1], need[2], ctx.wdtype) + (None,)


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               eps: float = 1e-5, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """(x - mean) / sqrt(variance + eps) * weight + bias over x's last axis,
    differentiable in x, weight and bias.  x: any contiguous tensor, or a
    two-dimensional one with neighbouring columns; weight and bias: x's dtype or
    float32.  ``out`` (which may be x) records no gradient, so with it none may
    be wanted."""
    if stream is not None:
        return _on(stream, layer_norm, x, weight, bias, eps, out)
    if isinstance(x, torch.Tensor) and _recorded(x, weight, bias):
        if out is not None:
            raise ValueError("out: a gradient is being recorded, and would be lost")
        return _Norm.apply(x, weight, bias, eps)
    return _norm(x, weight, bias, eps, out, False)[0]
