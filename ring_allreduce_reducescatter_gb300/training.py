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
    i64 = ctypes.c_longlong
    for f in ("ring_linear_cross_entropy_workspace", "ring_linear_cross_entropy_backward_workspace"):
        getattr(L, f).argtypes, getattr(L, f).restype = [vp, sz, vp, sz, sz, sz, sz], sz
    L.ring_linear_cross_entropy.argtypes = [vp, sz, vp, sz, vp, i64, vp, vp, vp, sz, sz, sz, i, vp, sz, vp]
    L.ring_linear_cross_entropy_backward.argtypes = [vp, sz, vp, sz, vp, sz, vp, i64, vp, vp, sz, vp, sz, sz, sz, sz, i, vp,
                                                     sz, vp]
    L.ring_orthogonalize_workspace.argtypes, L.ring_orthogonalize_workspace.restype = [sz, sz, sz], sz
    L.ring_orthogonalize.argtypes = [vp, sz, sz, i, vp, sz, sz, i, sz, sz, sz, i, f64, vp, sz, vp]
    for f in ("ring_layer_norm", "ring_layer_norm_backward", "ring_linear_cross_entropy", "ring_linear_cross_entropy_backward",
              "ring_orthogonalize"):
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


def _weights(x, cols, code, weight, bias):
    """The C code of the weights' one dtype (x's, ``code``, where there are none)."""
    wtype = None
    for name, t in (("weight", weight), ("bias", bias)):
        if t is None:
            continue
        if not isinstance(t, torch.Tensor) or t.shape != (cols,) or not t.is_contiguous() or t.device != x.device:
            raise ValueError(f"{name}: needs a contiguous tensor of {cols} elements on {x.device}")
        got = t.dtype
        if (got != x.dtype and got != _F32) or (wtype is not None and got != wtype):
            raise ValueError(f"{name}: {got}; the weights have one dtype, x's ({x.dtype}) or float32")
        wtype = got
    return code if wtype is None or wtype == x.dtype else 0


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
    wcode = _weights(x, cols, code, weight, bias)
    if out is None:
        out, ld_out = torch.empty(x.shape, dtype=x.dtype, device=device), cols
    else:
        _, _, ld_out = _rows(out, "out")
        if out.shape != x.shape or out.dtype != x.dtype or out.device != device:
            raise ValueError("x and out must have one shape, dtype and device")
    mean = rstd = None
    if stats:
        mean = torch.empty(x.shape[:-1], dtype=_F32, device=device)
        rstd = torch.empty_like(mean)
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
    for t in (mean, rstd):
        if (not isinstance(t, torch.Tensor) or t.dtype != _F32 or t.numel() != rows or t.device != device
                or not t.is_contiguous()):
            raise ValueError(f"mean and rstd: need contiguous float32 tensors of {rows} elements on {device}")
    code, handle = _dtype(x.dtype), _current(device)
    wcode, wtype = _weights(x, cols, code, weight, None), x.dtype
    if weight is not None:
        wtype = weight.dtype
    elif wdtype is not None and wdtype != wtype:
        if wdtype != _F32:
            raise ValueError(f"wdtype {wdtype}: x's dtype ({x.dtype}) or float32 is wanted")
        wtype, wcode = _F32, 0
    dx = torch.empty(x.shape, dtype=x.dtype, device=device) if want_dx else None
    dweight = torch.empty(cols, dtype=wtype, device=device) if want_dweight else None
    dbias = None if not want_dbias else torch.empty_like(dweight) if want_dweight else torch.empty(cols, dtype=wtype, device=device)
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


# ------------------------------------------------------- linear cross entropy


def _loss_operands(x, w, target):
    tokens, hidden, ld_x = _matrix(x, "x")
    vocabulary, h, ld_w = _matrix(w, "w")
    if h != hidden:
        raise ValueError(f"x has {hidden} columns, w {h}")
    if x.dtype != w.dtype or x.dtype not in (torch.float16, torch.bfloat16):
        raise ValueError(f"x is {x.dtype}, w {w.dtype}: both float16 or both bfloat16 are wanted")
    if (not isinstance(target, torch.Tensor) or target.dtype != torch.int64 or target.shape != (tokens,)
            or not target.is_contiguous()):
        raise ValueError(f"target: needs a contiguous int64 tensor of {tokens} elements")
    if w.device != x.device or target.device != x.device:
        raise ValueError("x, w and target must be on one device")
    if hidden < 1 or vocabulary < 1:
        raise ValueError("hidden size and vocabulary must not be empty")
    return tokens, hidden, vocabulary, max(ld_x, hidden), max(ld_w, hidden), _dtype(x.dtype)


def _losses(x, w, target, ignore_index, want_lse, want_sums):
    """(loss, lse, sums), None for what is not wanted."""
    tokens, hidden, vocabulary, ld_x, ld_w, code = _loss_operands(x, w, target)
    device, handle, L = x.device, _current(x.device), _L or _lib()
    loss = torch.empty(tokens, dtype=_F32, device=device)
    lse = torch.empty_like(loss) if want_lse else None
    sums = torch.empty(3, dtype=_F32, device=device) if want_sums else None
    at = (x.data_ptr(), ld_x, w.data_ptr(), ld_w)
    need = L.ring_linear_cross_entropy_workspace(*at, tokens, hidden, vocabulary)
    space = torch.empty(need, dtype=torch.uint8, device=device)
    status = L.ring_linear_cross_entropy(*at, target.data_ptr(), ignore_index, loss.data_ptr(), _at(lse), _at(sums), tokens,
                                         hidden, vocabulary, code, space.data_ptr(), need, handle)
    if status:
        _failed(status, "ring_linear_cross_entropy")
    return loss, lse, sums


def linear_cross_entropy_forward(x: torch.Tensor, w: torch.Tensor, target: torch.Tensor, ignore_index: int = -100,
                                 stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(loss, lse) of every token, float32: the softmax cross entropy of the
    logits x @ w.T, which are never stored, against target, and the logarithm of
    the sum of their exponentials, as linear_cross_entropy_backward takes it.
    Records no gradient (linear_cross_entropy does)."""
    if stream is not None:
        return _on(stream, linear_cross_entropy_forward, x, w, target, ignore_index)
    if _recorded(x, w):
        raise ValueError("a gradient is being recorded, and would be lost: linear_cross_entropy records it")
    return _losses(x, w, target, ignore_index, True, False)[:2]


def linear_cross_entropy_backward(grad: torch.Tensor, x: torch.Tensor, w: torch.Tensor, target: torch.Tensor,
                                  lse: torch.Tensor, ignore_index: int = -100, want_dx: bool = True, want_dw: bool = True,
                                  stream=None) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """(dx, dw) for the gradient of the tokens' losses: grad, float32, one element
    for all tokens or one each.  None for what is not wanted."""
    if stream is not None:
        return _on(stream, linear_cross_entropy_backward, grad, x, w, target, lse, ignore_index, want_dx, want_dw)
    tokens, hidden, vocabulary, ld_x, ld_w, code = _loss_operands(x, w, target)
    device = x.device
    if (not isinstance(grad, torch.Tensor) or grad.dtype != _F32 or grad.device != device or not grad.is_contiguous()
            or not (grad.numel() == 1 or grad.shape == (tokens,))):
        raise ValueError(f"grad: needs a contiguous float32 tensor of one element or of {tokens} on {device}")
    if (not isinstance(lse, torch.Tensor) or lse.dtype != _F32 or lse.device != device or lse.shape != (tokens,)
            or not lse.is_contiguous()):
        raise ValueError(f"lse: needs a contiguous float32 tensor of {tokens} elements on {device}")
    handle, L = _current(device), _L or _lib()
    dx = torch.empty((tokens, hidden), dtype=x.dtype, device=device) if want_dx else None
    dw = torch.empty((vocabulary, hidden), dtype=x.dtype, device=device) if want_dw else None
    at = (x.data_ptr(), ld_x, w.data_ptr(), ld_w)
    need = L.ring_linear_cross_entropy_backward_workspace(*at, tokens, hidden, vocabulary)
    space = torch.empty(need, dtype=torch.uint8, device=device)
    status = L.ring_linear_cross_entropy_backward(grad.data_ptr(), 0 if grad.numel() == 1 else 1, *at, target.data_ptr(),
                                                  ignore_index, lse.data_ptr(), _at(dx), hidden, _at(dw), hidden, tokens, hidden,
                                                  vocabulary, code, space.data_ptr(), need, handle)
    if status:
        _failed(status, "ring_linear_cross_entropy_backward")
    return dx, dw


_REDUCTIONS = {"none": None, "sum": 0, "mean": 2}


class _CrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, target, ignore_index, reduction):
        loss, lse, sums = _losses(x, w, target, ignore_index, True, reduction != "none")
        ctx.save_for_backward(x, w, target, lse, sums)
        ctx.ignore_index, ctx.reduction = ignore_index, reduction
        return loss if sums is None else sums[_REDUCTIONS[reduction]].clone()

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, w, target, lse, sums = ctx.saved_tensors
        grad = dy.contiguous()
        if ctx.reduction == "mean":
            grad = grad / sums[1].clamp(min=1)
        need = ctx.needs_input_grad
        return linear_cross_entropy_backward(grad, x, w, target, lse, ctx.ignore_index, need[0], need[1]) + (None, None, None)


def linear_cross_entropy(x: torch.Tensor, w: torch.Tensor, target: torch.Tensor, ignore_index: int = -100,
                         reduction: str = "mean", stream=None) -> torch.Tensor:
    """The softmax cross entropy of the logits x @ w.T (x: [tokens, hidden], w:
    [vocabulary, hidden], float16 or bfloat16) against target (int64, one a
    token), differentiable in x and w; neither the logits nor their gradient is
    ever stored whole.  A token whose target is ignore_index counts nothing.
    reduction: "mean" over the tokens that count (0 if none does), "sum", or
    "none" (each token's, 0 for one that does not count); float32."""
    if reduction not in _REDUCTIONS:
        raise ValueError(f"reduction {reduction!r}: 'mean', 'sum' or 'none' is wanted")
    if stream is not None:
        return _on(stream, linear_cross_entropy, x, w, target, ignore_index, reduction)
    if isinstance(x, torch.Tensor) and isinstance(w, torch.Tensor) and _recorded(x, w):
        return _CrossEntropy.apply(x, w, target, ignore_index, reduction)
    loss, _, sums = _losses(x, w, target, ignore_index, False, reduction != "none")
    return loss if sums is None else sums[_REDUCTIONS[reduction]]


# -------------------------------------------------------- orthogonalised update


def _batch(t, name):
    """(batch, rows, cols, row stride, matrix stride) of one matrix or a batch of
    them, with neighbouring columns."""
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dim() == 3:
        b, m, n = t.shape
        if t.numel() == 0:
            return b, m, n, n, m * n
        _, _, ld = _matrix(t[0], name)
        if b > 1 and t.stride(0) < (m - 1) * ld + n:
            raise ValueError(f"{name}: the matrices of a batch must not overlap")
        return b, m, n, ld, t.stride(0)
    m, n, ld = _matrix(t, name)
    return 1, m, n, ld, 0


def orthogonalize(g: torch.Tensor, steps: int = 5, eps: float = 1e-7, dtype: Optional[torch.dtype] = None,
                  out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The matrix g, or each of a batch [batch, rows, cols], brought near the
    orthogonal matrix that has its singular vectors by Newton-Schulz steps with
    the coefficients (3.4445, -4.7750, 2.0315), which take every singular value
    to about one; the step of the Muon optimiser, for the sum of the ranks'
    gradients.  dtype: of the result (g's if None, or that of ``out``, which may
    be g).  Records no gradient, so none may be wanted of g."""
    if stream is not None:
        return _on(stream, orthogonalize, g, steps, eps, dtype, out)
    b, m, n, ld, stride = _batch(g, "g")
    if _recorded(g):
        raise ValueError("g: a gradient is being recorded, and would be lost")
    code, device, handle = _dtype(g.dtype), g.device, _current(g.device)
    if out is None:
        out = torch.empty(g.shape, dtype=g.dtype if dtype is None else dtype, device=device)
        ld_out, stride_out = n, m * n
    else:
        if not isinstance(out, torch.Tensor) or out.shape != g.shape or out.device != device:
            raise ValueError("out must have g's shape and device")
        if dtype not in (None, out.dtype):
            raise ValueError(f"out: {out.dtype}, expected {dtype}")
        _, _, _, ld_out, stride_out = _batch(out, "out")
    out_code = _dtype(out.dtype)
    L = _L or _lib()
    need = L.ring_orthogonalize_workspace(b, m, n)
    space = torch.empty(need, dtype=torch.uint8, device=device)
    status = L.ring_orthogonalize(g.data_ptr(), ld, stride, code, out.data_ptr(), ld_out, stride_out, out_code, b, m, n, steps,
                                  eps, space.data_ptr(), need, handle)
    if status:
        _failed(status, "ring_orthogonalize")
    return out
