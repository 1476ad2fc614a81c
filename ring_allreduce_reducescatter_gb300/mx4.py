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


def _check(status: int, what: str) -> None:
    if status:
        from . import RingError

        raise RingError(status, what)


class Mx4:
    """A rows x cols matrix in microscaled 4 bits: ``data``, uint8
    [rows, 16 * ceil(cols / 32)], and ``scales``, uint8
    [ceil(rows / 128), ceil(cols / 256), 1024]."""

    __slots__ = ("data", "scales", "rows", "cols", "_c", "_at")

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
        self._set(data, scales, rows, cols)

    def _set(self, data, scales, rows, cols):
        self.data, self.scales, self.rows, self.cols = data, scales, rows, cols
        self._c = _Matrix(data.data_ptr(), scales.data_ptr(), rows, cols)
        self._at = ctypes.addressof(self._c)
        return self

    @classmethod
    def empty(cls, rows: int, cols: int, device=None) -> "Mx4":
        """A matrix whose bytes are not set yet."""
        if rows < 0 or cols < 0:
            raise ValueError("rows and cols must not be negative")
        device = torch.device("cuda") if device is None else device
        return cls.__new__(cls)._set(
            torch.empty((rows, -(-cols // 32) * 16), dtype=torch.uint8, device=device),
            torch.empty((-(-rows // 128), -(-cols // 256), 1024), dtype=torch.uint8, device=device), rows, cols)

    @property
    def shape(self) -> Tuple[int, int]:
        return self.rows, self.cols

    @property
    def device(self):
        return self.data.device

    def _tensors(self):
        return self.data, self.scales

    def __repr__(self):
        return f"Mx4({self.rows} x {self.cols}, {self.data.device})"


class _On:
    """The stream of one call: its handle, allocation on it, and the record
    that keeps the call's tensors alive on it when it is not the current one."""

    __slots__ = ("handle", "_stream", "_outer")

    def __init__(self, device, stream):
        if device.index is not None and device.index != torch.cuda.current_device():
            raise ValueError(f"the tensors are on {device}, the current device is cuda:{torch.cuda.current_device()}")
        self._outer = self._stream = None
        if stream is None:
            self.handle = torch.cuda.current_stream().cuda_stream or None
            return
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()
        self.handle = stream.cuda_stream or None
        if stream != torch.cuda.current_stream():
            self._stream = stream

    def __enter__(self):
        if self._stream is not None:
            self._outer = torch.cuda.stream(self._stream)
            self._outer.__enter__()
        return self

    def __exit__(self, *exc):
        if self._outer is not None:
            self._outer.__exit__(*exc)

    def used(self, *tensors):
        if self._stream is not None:
            for t in tensors:
                if t is not None:
                    for u in t._tensors() if isinstance(t, Mx4) else (t,):
                        u.record_stream(self._stream)


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


def _quantize(x, want_rows, want_cols, rounding, seed, subsequence, dropout, out_rows, out_cols, stream):
    rows, cols, ld = _matrix(x, "x")
    code = _dtype(x.dtype)
    try:
        how = _ROUNDING[rounding]
    except KeyError:
        raise ValueError(f"rounding {rounding!r}: 'nearest' or 'stochastic' is wanted") from None
    with _On(x.device, stream) as on:
        if want_rows and out_rows is None:
            out_rows = Mx4.empty(rows, cols, x.device)
        if want_cols and out_cols is None:
            out_cols = Mx4.empty(cols, rows, x.device)
        for q in (out_rows, out_cols):
            if q is not None and q.device != x.device:
                raise ValueError(f"out is on {q.device}, x on {x.device}")
        _check(_lib().ring_mx4_quantize(x.data_ptr(), rows, cols, ld, code, out_rows and out_rows._at,
                                        out_cols and out_cols._at, how, seed & _U64, subsequence & _U64,
                                        _drop(dropout), on.handle), "ring_mx4_quantize")
        on.used(x, out_rows, out_cols)
    return out_rows, out_cols


def mx4_quantize(x: torch.Tensor, transposed: bool = False, rounding: str = "nearest", seed: int = 0,
                 subsequence: int = 0, dropout: Optional[Dropout] = None, out: Optional[Mx4] = None,
                 stream=None) -> Mx4:
    """x (two dimensions) in 4 bits along its rows; transposed: the transpose
    of x, along its own rows (x's columns).  dropout is applied to x first."""
    if transposed:
        return _quantize(x, False, True, rounding, seed, subsequence, dropout, None, out, stream)[1]
    return _quantize(x, True, False, rounding, seed, subsequence, dropout, out, None, stream)[0]


def mx4_quantize_both(x: torch.Tensor, rounding: str = "nearest", seed: int = 0, subsequence: int = 0,
                      dropout: Optional[Dropout] = None, stream=None) -> Tuple[Mx4, Mx4]:
    """x and its transpose in 4 bits, x read once (stochastic rounding of the
    transpose takes subsequence + 1)."""
    return _quantize(x, True, True, rounding, seed, subsequence, dropout, None, None, stream)


def mx4_dequantize(q: Mx4, dtype: torch.dtype = torch.float32, out: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """The values of a 4-bit matrix, rounded to dtype (exact in binary32 and
    bfloat16, but 4 and 6 times 2^126, which lie above both: infinity)."""
    with _On(q.device, stream) as on:
        if out is None:
            out = torch.empty((q.rows, q.cols), dtype=dtype, device=q.device)
            ld = q.cols
        else:
            ld = _output(out, q.rows, q.cols, q.device)
        _check(_lib().ring_mx4_dequantize(q._at, out.data_ptr(), ld, _dtype(out.dtype), on.handle),
               "ring_mx4_dequantize")
        on.used(q, out)
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
    dtype (that of ``out`` if it is given) and may be ``out`` itself."""
    if a.cols != b.cols:
        raise ValueError(f"a has {a.cols} columns, b {b.cols}")
    m, n, device = a.rows, b.rows, a.device
    if b.device != device:
        raise ValueError(f"a is on {device}, b on {b.device}")
    ld_res, res = 0, None
    with _On(device, stream) as on:
        if out is None:
            out = torch.empty((m, n), dtype=dtype, device=device)
            ld = n
        else:
            ld = _output(out, m, n, device)
        if residual is not None:
            ld_res, res = _output(residual, m, n, device, "residual"), residual.data_ptr()
            if residual.dtype != out.dtype:
                raise ValueError(f"residual: {residual.dtype}, the output is {out.dtype}")
        _check(_lib().ring_mx4_matmul(a._at, b._at, out.data_ptr(), ld, _dtype(out.dtype), res, ld_res,
                                      _drop(dropout), on.handle), "ring_mx4_matmul")
        on.used(a, b, residual, out)
    return out


def dropout(x: torch.Tensor, drop: Dropout, residual: Optional[torch.Tensor] = None,
            out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """(residual +) dropout(x).  The backward pass is dropout(dy, drop) with the
    same ``drop``.  Contiguous tensors of any shape, or two-dimensional views
    with neighbouring columns."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError("x: needs a CUDA tensor")
    code = _dtype(x.dtype)
    with _On(x.device, stream) as on:
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        ts = (x, out) if residual is None else (x, out, residual)
        if any(t.shape != x.shape or t.dtype != x.dtype or t.device != x.device for t in ts):
            raise ValueError("x, residual and out must have one shape, dtype and device")
        if x.is_contiguous() and out.is_contiguous() and (residual is None or residual.is_contiguous()):
            rows, cols = 1, x.numel()
            lds = [cols] * 3
        else:
            rows, cols = _matrix(x, "x")[:2]
            lds = [_matrix(t, "x, residual and out")[2] for t in ts] + [cols]
        _check(_lib().ring_dropout(x.data_ptr(), lds[0], None if residual is None else residual.data_ptr(),
                                   lds[2], out.data_ptr(), lds[1], rows, cols, code, _drop(drop), on.handle),
               "ring_dropout")
        on.used(*ts)
    return out


def mx4_allreduce(qs: Sequence[Mx4], outs: Optional[Sequence[torch.Tensor]] = None,
                  dtype: torch.dtype = torch.float32, stream=None):
    """The flat ring's AllReduce of R equal 4-bit matrices: every output holds
    the binary32 fold of their values, rounded once to its dtype."""
    qs = list(qs)
    if not qs:
        raise ValueError("qs: need at least one rank")
    R, shape, device = len(qs), qs[0].shape, qs[0].device
    if any(q.shape != shape or q.device != device for q in qs):
        raise ValueError("qs: every rank's matrix must have one shape and device")
    with _On(device, stream) as on:
        if outs is None:
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
        _check(_lib().ring_mx4_allreduce(mats, ptrs, R, _dtype(outs[0].dtype), on.handle), "ring_mx4_allreduce")
        on.used(*qs, *outs)
    return outs


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, residual, drop, seed, subsequence):
        x_rows, x_cols = mx4_quantize_both(x)
        w_rows, w_cols = mx4_quantize_both(w)
        ctx.kept = x_cols, w_cols, drop, seed, subsequence
        ctx.has_residual = residual is not None
        return mx4_matmul(x_rows, w_rows, x.dtype, residual=residual, dropout=drop)

    @staticmethod
    def backward(ctx, dy):
        x_cols, w_cols, drop, seed, subsequence = ctx.kept
        if dy.stride(1) != 1 or dy.stride(0) < dy.shape[1]:
            dy = dy.contiguous()
        g_rows, g_cols = mx4_quantize_both(dy, "stochastic", seed, subsequence, dropout=drop)
        dx = mx4_matmul(g_rows, w_cols, dy.dtype) if ctx.needs_input_grad[0] else None
        dw = mx4_matmul(g_cols, x_cols, dy.dtype) if ctx.needs_input_grad[1] else None
        return dx, dw, dy if ctx.has_residual else None, None, None, None


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
    return _Linear.apply(x, w, residual, drop, seed, subsequence)
