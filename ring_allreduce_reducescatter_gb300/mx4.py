"""Microscaled 4-bit matrices, their products and AllReduce, and dropout.

The binding of the ``ring_mx4_*`` and ``ring_dropout`` entry points of
``include/ringred.h`` (which defines the format, the rounding and the random
numbers), and ``mx4_linear``, the linear layer of 4-bit training made of them.
As elsewhere in the package only arguments are marshalled here; outputs that
are not given are torch tensors allocated on the stream of the call.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional, Sequence, Tuple

import torch

NEAREST, STOCHASTIC = 0, 1
_ROUNDING = {"nearest": NEAREST, "stochastic": STOCHASTIC}
_DTYPE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_U64 = (1 << 64) - 1


class _Matrix(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("rows", ctypes.c_size_t),
                ("cols", ctypes.c_size_t)]


class _Drop(ctypes.Structure):
    _fields_ = [("p", ctypes.c_double), ("seed", ctypes.c_ulonglong), ("subsequence", ctypes.c_ulonglong),
                ("first", ctypes.c_ulonglong)]


class Dropout(NamedTuple):
    """Which elements are dropped: probability p (held to 1 / 65536), the
    generator's seed and subsequence, and the index of the tensor's first
    element (for a shard or a range of a larger tensor)."""

    p: float
    seed: int
    subsequence: int = 0
    first: int = 0


def bind(L) -> None:
    """Argument types of the entry points, called once when the library loads."""
    sz, i, vp, u64 = ctypes.c_size_t, ctypes.c_int, ctypes.c_void_p, ctypes.c_ulonglong
    L.ring_mx4_row_bytes.argtypes, L.ring_mx4_row_bytes.restype = [sz], sz
    L.ring_mx4_scale_bytes.argtypes, L.ring_mx4_scale_bytes.restype = [sz, sz], sz
    L.ring_mx4_quantize.argtypes = [vp, sz, sz, sz, i, vp, vp, i, u64, u64, vp, vp]
    L.ring_mx4_dequantize.argtypes = [vp, vp, sz, i, vp]
    L.ring_mx4_matmul.argtypes = [vp, vp, vp, sz, i, vp, sz, vp, vp]
    L.ring_dropout.argtypes = [vp, sz, vp, sz, vp, sz, sz, sz, i, vp, vp]
    L.ring_mx4_allreduce.argtypes = [ctypes.POINTER(_Matrix), ctypes.POINTER(vp), i, i, vp]
    for f in ("ring_mx4_quantize", "ring_mx4_dequantize", "ring_mx4_matmul", "ring_dropout", "ring_mx4_allreduce"):
        getattr(L, f).restype = i


_L = None


def _lib():
    global _L
    if _L is None:
        from . import lib

        _L = lib()
    return _L


def _failed(status: int, what: str):
    from . import RingError

    raise RingError(status, what)


class Mx4:
    """A rows x cols matrix in microscaled 4 bits: ``data``, uint8
    [rows, 16 * ceil(cols / 32)], and ``scales``, uint8
    [ceil(rows / 128), ceil(cols / 256), 1024]."""

    __slots__ = ("rows", "cols", "device", "_data", "_scales", "_whole", "_c", "_at")

    def __init__(self, data: torch.Tensor, scales: torch.Tensor, rows: int, cols: int):
        if rows < 0 or cols < 0:
            raise ValueError("rows and cols must not be negative")
        for name, t, n in (("data", data, rows * (-(-cols // 32) * 16)),
                           ("scales", scales, -(-rows // 128) * (-(-cols // 256) * 1024))):
            if t.dtype != torch.uint8 or not t.is_cuda or not t.is_contiguous():
                raise ValueError(f"{name}: needs a contiguous CUDA tensor of uint8")
            if t.numel() != n:
                raise ValueError(f"{name}: {t.numel()} bytes, expected {n} for {rows} x {cols}")
        if scales.device != data.device:
            raise ValueError("data and scales must be on one device")
        self.rows, self.cols, self.device = rows, cols, data.device
        self._data, self._scales, self._whole = data, scales, None
        self._c = _Matrix(data.data_ptr(), scales.data_ptr(), rows, cols)
        self._at = ctypes.addressof(self._c)

    @classmethod
    def empty(cls, rows: int, cols: int, device=None) -> "Mx4":
        """A matrix whose bytes are not set yet, in one allocation."""
        if rows < 0 or cols < 0:
            raise ValueError("rows and cols must not be negative")
        return _new(rows, cols, "cuda" if device is None else device)

    @property
    def data(self) -> torch.Tensor:
        if self._whole is not None:
            self._split()
        return self._data

    @property
    def scales(self) -> torch.Tensor:
        if self._whole is not None:
            self._split()
        return self._scales

    def _split(self):
        n, whole = self._scales, self._whole
        self._data = whole[:n].view(self.rows, -(-self.cols // 32) * 16)
        self._scales = whole[n:].view(-(-self.rows // 128), -(-self.cols // 256), 1024)
        self._whole = None

    @property
    def shape(self) -> Tuple[int, int]:
        return self.rows, self.cols

    def __repr__(self):
        return f"Mx4({self.rows} x {self.cols}, {self.device})"


def _new(rows, cols, device) -> Mx4:
    """Mx4.empty without its checks."""
    n = rows * ((cols + 31) // 32 * 16)
    whole = torch.empty(n + (rows + 127) // 128 * ((cols + 255) // 256 * 1024), dtype=torch.uint8, device=device)
    return _of(whole, n, rows, cols)


def _of(whole, n, rows, cols) -> Mx4:
    """The matrix whose bytes are those of `whole`: n of data, then the scales."""
    q = Mx4.__new__(Mx4)
    at = whole.data_ptr()
    q.rows, q.cols, q.device = rows, cols, whole.device
    q._data, q._scales, q._whole = None, n, whole
    q._c = c = _Matrix(at, at + n, rows, cols)
    q._at = ctypes.addressof(c)
    return q


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _current(device):
    """The handle of the device's current stream; the device must be the current one."""
    at = torch.cuda.current_device()
    if device.index != at:
        raise ValueError(f"the tensors are on {device}, the current device is cuda:{at}")
    return (_raw_stream(at) if _raw_stream is not None else torch.cuda.current_stream().cuda_stream) or None


def _on(stream, call, *args):
    """call(*args) with `stream` current, so that its outputs are allocated for
    that stream, and its tensors kept from reuse until the stream is past it."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()
    with torch.cuda.stream(stream):
        out = call(*args)
    for t in args + (out if isinstance(out, tuple) else (out,)):
        for u in t if isinstance(t, (list, tuple)) else (t,):
            if isinstance(u, Mx4):
                for part in (u._whole,) if u._whole is not None else (u._data, u._scales):
                    part.record_stream(stream)
            elif isinstance(u, torch.Tensor):
                u.record_stream(stream)
    return out


def _dtype(t: torch.dtype) -> int:
    try:
        return _DTYPE[t]
    except KeyError:
        raise ValueError(f"dtype {t}: float32, float16 or bfloat16 is wanted") from None


def _matrix(t, name: str):
    """(rows, cols, row stride) of a two-dimensional CUDA tensor with neighbouring columns."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name}: needs a CUDA tensor")
    if t.dim() != 2:
        raise ValueError(f"{name}: needs two dimensions, got {t.dim()}")
    rows, cols = t.shape
    ld, step = t.stride()
    if (step != 1 and cols > 1) or (ld < cols and rows > 1):
        raise ValueError(f"{name}: the elements of a row must follow one another and rows must not overlap")
    return rows, cols, ld if rows > 1 else cols


def _drop(d: Optional[Dropout]):
    if d is None:
        return None
    return ctypes.byref(_Drop(d.p, d.seed & _U64, d.subsequence & _U64, d.first & _U64))


def _quantize(x, want_rows, want_cols, rounding, seed, subsequence, dropout, out_rows, out_cols):
    rows, cols, ld = _matrix(x, "x")
    device = x.device
    handle = _current(device)
    code = _dtype(x.dtype)
    how = _ROUNDING.get(rounding)
    if how is None:
        raise ValueError(f"rounding {rounding!r}: 'nearest' or 'stochastic' is wanted")
    for q in (out_rows, out_cols):
        if q is not None and q.device != device:
            raise ValueError(f"out is on {q.device}, x on {device}")
    by_rows = by_cols = None
    if want_rows:
        if out_rows is None:
            out_rows = _new(rows, cols, device)
        by_rows = out_rows._at
    if want_cols:
        if out_cols is None:
            out_cols = _new(cols, rows, device)
        by_cols = out_cols._at
    status = (_L or _lib()).ring_mx4_quantize(x.data_ptr(), rows, cols, ld, code, by_rows, by_cols, how, seed & _U64,
                                              subsequence & _U64, _drop(dropout), handle)
    if status:
        _failed(status, "ring_mx4_quantize")
    return out_rows, out_cols


def mx4_quantize(x: torch.Tensor, transposed: bool = False, rounding: str = "nearest", seed: int = 0,
                 subsequence: int = 0, dropout: Optional[Dropout] = None, out: Optional[Mx4] = None,
                 stream=None) -> Mx4:
    """x (two dimensions) in 4 bits along its rows; transposed: the transpose
    of x, along its own rows (x's columns).  dropout is applied to x first."""
    if stream is not None:
        return _on(stream, mx4_quantize, x, transposed, rounding, seed, subsequence, dropout, out)
    if transposed:
        return _quantize(x, False, True, rounding, seed, subsequence, dropout, None, out)[1]
    return _quantize(x, True, False, rounding, seed, subsequence, dropout, out, None)[0]


def mx4_quantize_both(x: torch.Tensor, rounding: str = "nearest", seed: int = 0, subsequence: int = 0,
                      dropout: Optional[Dropout] = None, stream=None) -> Tuple[Mx4, Mx4]:
    """x and its transpose in 4 bits, x read once (stochastic rounding of the
    transpose takes subsequence + 1)."""
    if stream is not None:
        return _on(stream, mx4_quantize_both, x, rounding, seed, subsequence, dropout)
    return _quantize(x, True, True, rounding, seed, subsequence, dropout, None, None)


def mx4_dequantize(q: Mx4, dtype: torch.dtype = torch.float32, out: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """The values of a 4-bit matrix, rounded to dtype (exact in binary32 and
    bfloat16, but 4 and 6 times 2^126, which lie above both: infinity)."""
    if stream is not None:
        return _on(stream, mx4_dequantize, q, dtype, out)
    handle = _current(q.device)
    if out is None:
        code = _dtype(dtype)
        out, ld = torch.empty((q.rows, q.cols), dtype=dtype, device=q.device), q.cols
    else:
        code, ld = _dtype(out.dtype), _output(out, q.rows, q.cols, q.device)
    status = (_L or _lib()).ring_mx4_dequantize(q._at, out.data_ptr(), ld, code, handle)
    if status:
        _failed(status, "ring_mx4_dequantize")
    return out


def _output(out, rows, cols, device, name="out"):
    r, c, ld = _matrix(out, name)
    if (r, c) != (rows, cols):
        raise ValueError(f"{name}: {r} x {c}, expected {rows} x {cols}")
    if out.device != device:
        raise ValueError(f"{name}: on {out.device}, expected {device}")
    return ld


def mx4_matmul(a: Mx4, b: Mx4, dtype: torch.dtype = torch.bfloat16, residual: Optional[torch.Tensor] = None,
               dropout: Optional[Dropout] = None, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """(residual +) dropout(a @ b.T), a.rows x b.rows; residual has the output's
    dtype (that of ``out`` if it is given) and may be ``out`` itself.
    Differentiable in residual (4-bit matrices hold no gradient: mx4_linear is
    the layer that has one); with ``out``, none may be wanted."""
    if stream is not None:
        return _on(stream, mx4_matmul, a, b, dtype, residual, dropout, out)
    if isinstance(residual, torch.Tensor) and residual.requires_grad and torch.is_grad_enabled():
        if out is not None:
            raise ValueError("out: a gradient of residual is being recorded, and would be lost")
        return _OntoResidual.apply(residual, a, b, dtype, dropout)
    if a.cols != b.cols:
        raise ValueError(f"a has {a.cols} columns, b {b.cols}")
    m, n, device = a.rows, b.rows, a.device
    if b.device != device:
        raise ValueError(f"a is on {device}, b on {b.device}")
    handle = _current(device)
    if out is None:
        code = _dtype(dtype)
        out, ld = torch.empty((m, n), dtype=dtype, device=device), n
    else:
        code, ld = _dtype(out.dtype), _output(out, m, n, device)
    ld_res, res = 0, None
    if residual is not None:
        ld_res, res = _output(residual, m, n, device, "residual"), residual.data_ptr()
        if residual.dtype != out.dtype:
            raise ValueError(f"residual: {residual.dtype}, the output is {out.dtype}")
    status = (_L or _lib()).ring_mx4_matmul(a._at, b._at, out.data_ptr(), ld, code, res, ld_res, _drop(dropout), handle)
    if status:
        _failed(status, "ring_mx4_matmul")
    return out


class _OntoResidual(torch.autograd.Function):
    @staticmethod
    def forward(ctx, residual, a, b, dtype, drop):
        return mx4_matmul(a, b, dtype, residual, drop)

    @staticmethod
    def backward(ctx, dy):
        return dy, None, None, None, None


def dropout(x: torch.Tensor, drop: Dropout, residual: Optional[torch.Tensor] = None,
            out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """(residual +) dropout(x), differentiable in x and residual (the backward
    pass is dropout(dy, drop) with the same ``drop``).  Contiguous tensors of
    any shape, or two-dimensional views with neighbouring columns.  ``out``
    records no gradient, so with it none may be wanted of x or residual."""
    if stream is not None:
        return _on(stream, _dropout, x, drop, residual, out)
    return _dropout(x, drop, residual, out)


class _Dropped(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, drop):
        ctx.drop = drop
        return _dropout(x, drop, residual, None)  # (nothing is recorded in here)

    @staticmethod
    def backward(ctx, dy):
        # (the mask goes by the index in row-major order, whatever dy's layout)
        dx = _dropout(dy.contiguous(), ctx.drop, None, None) if ctx.needs_input_grad[0] else None
        return dx, dy if ctx.needs_input_grad[1] else None, None


def _dropout(x, drop, residual, out):
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError("x: needs a CUDA tensor")
    if (x.requires_grad or (residual is not None and residual.requires_grad)) and torch.is_grad_enabled():
        if out is not None:
            raise ValueError("out: a gradient of x or residual is being recorded, and would be lost")
        return _Dropped.apply(x, residual, drop)
    device, flat = x.device, x.is_contiguous()
    code, handle = _dtype(x.dtype), _current(device)
    for t in (out, residual):
        if t is not None:
            if t.shape != x.shape or t.dtype != x.dtype or t.device != device:
                raise ValueError("x, residual and out must have one shape, dtype and device")
            flat = flat and t.is_contiguous()
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=device)
    if flat:
        rows, ld_x = 1, x.numel()
        cols = ld_out = ld_res = ld_x
    else:
        rows, cols, ld_x = _matrix(x, "x")
        ld_out = _matrix(out, "out")[2]
        ld_res = cols if residual is None else _matrix(residual, "residual")[2]
    status = (_L or _lib()).ring_dropout(x.data_ptr(), ld_x, None if residual is None else residual.data_ptr(), ld_res,
                                         out.data_ptr(), ld_out, rows, cols, code, _drop(drop), handle)
    if status:
        _failed(status, "ring_dropout")
    return out


def mx4_allreduce(qs: Sequence[Mx4], outs: Optional[Sequence[torch.Tensor]] = None,
                  dtype: torch.dtype = torch.float32, stream=None):
    """The flat ring's AllReduce of R equal 4-bit matrices: every output holds
    the binary32 fold of their values, rounded once to its dtype."""
    if stream is not None:
        return _on(stream, mx4_allreduce, list(qs), None if outs is None else list(outs), dtype)
    qs = list(qs)
    if not qs:
        raise ValueError("qs: need at least one rank")
    R, shape, device = len(qs), qs[0].shape, qs[0].device
    if any(q.rows != shape[0] or q.cols != shape[1] or q.device != device for q in qs):
        raise ValueError("qs: every rank's matrix must have one shape and device")
    handle = _current(device)
    if outs is None:
        _dtype(dtype)
        outs = [torch.empty(shape, dtype=dtype, device=device) for _ in qs]
    else:
        outs = list(outs)
        if len(outs) != R:
            raise ValueError("qs and outs must have one matrix per rank")
        for t in outs:
            if (not isinstance(t, torch.Tensor) or tuple(t.shape) != shape or t.dtype != outs[0].dtype
                    or t.device != device or not t.is_contiguous()):
                raise ValueError("outs: contiguous tensors of the matrices' shape and device and one dtype are wanted")
    mats = (_Matrix * R)(*[q._c for q in qs])
    ptrs = (ctypes.c_void_p * R)(*[t.data_ptr() for t in outs])
    status = (_L or _lib()).ring_mx4_allreduce(mats, ptrs, R, _dtype(outs[0].dtype), handle)
    if status:
        _failed(status, "ring_mx4_allreduce")
    return outs


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, residual, drop, seed, subsequence, want_dx, want_dw):
        # a transpose is kept for the product of the backward pass that reads it
        x_rows, x_cols = mx4_quantize_both(x) if want_dw else (mx4_quantize(x), None)
        w_rows, w_cols = mx4_quantize_both(w) if want_dx else (mx4_quantize(w), None)
        # as saved tensors (their bytes): released with the graph, and seen by saved-tensor hooks
        kept = [q for q in (x_cols, w_cols) if q is not None]
        ctx.save_for_backward(*[q._whole for q in kept])
        ctx.sizes = [(q._scales, q.rows, q.cols) for q in kept]
        ctx.drop, ctx.seed, ctx.subsequence = drop, seed, subsequence
        ctx.want_dx, ctx.want_dw, ctx.has_residual = want_dx, want_dw, residual is not None
        return mx4_matmul(x_rows, w_rows, x.dtype, residual=residual, dropout=drop)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        want_dx, want_dw, drop, seed, subsequence = ctx.want_dx, ctx.want_dw, ctx.drop, ctx.seed, ctx.subsequence
        dx = dw = None
        if want_dx or want_dw:
            kept = [_of(whole, *size) for whole, size in zip(ctx.saved_tensors, ctx.sizes)]
            g = dy if dy.stride(1) == 1 and dy.stride(0) >= dy.shape[1] else dy.contiguous()
            # (each rounding keeps its numbers whether or not the other is wanted)
            if not want_dw:
                g_rows = mx4_quantize(g, False, "stochastic", seed, subsequence, drop)
            elif not want_dx:
                g_cols = mx4_quantize(g, True, "stochastic", seed, subsequence + 1, drop)
            else:
                g_rows, g_cols = mx4_quantize_both(g, "stochastic", seed, subsequence, drop)
            if want_dx:
                dx = mx4_matmul(g_rows, kept[-1], dy.dtype)
            if want_dw:
                dw = mx4_matmul(g_cols, kept[0], dy.dtype)
        return dx, dw, dy if ctx.has_residual else None, None, None, None, None, None


def mx4_linear(x: torch.Tensor, w: torch.Tensor, residual: Optional[torch.Tensor] = None,
               drop: Optional[Dropout] = None, seed: int = 0, subsequence: int = 0) -> torch.Tensor:
    """residual + dropout(x @ w.T) with the product, and both products of the
    backward pass, in 4 bits (differentiable in x, w and residual; 4-bit
    rounding counts as the identity).  x: [tokens, in], w: [out, in], one dtype.
    The gradient is rounded stochastically with the generator's subsequences
    ``subsequence`` and ``subsequence + 1`` of ``seed``; use fresh ones, other
    than the dropout's, every step."""
    if x.dtype != w.dtype or (residual is not None and residual.dtype != x.dtype):
        raise ValueError("x, w and residual must have one dtype")
    grad = torch.is_grad_enabled()
    return _Linear.apply(x, w, residual, drop, seed, subsequence, grad and x.requires_grad, grad and w.requires_grad)
