"""The microscaled linear layer on torch tensors.

``MXMatrix`` owns the codes and scales of a matrix in a microscaled format
(see "microscaled matrices" in ``include/q4adamw.h``); the functions allocate
results and workspaces with torch and forward to the ``q4mx_*`` calls.  They
compute nothing themselves.

A linear layer beside ``Q4State``, for a master stored [in, out]::

    w = mx.quantize(master, "fp4", transpose=True)       # after every step
    xq = mx.quantize(x, "fp8")                           # kept for backward
    y = mx.linear(xq, w)
    ...
    dx = mx.linear_dgrad(dy, w)
    mx.linear_wgrad(dy, xq, out=grad, transposed=True)   # the BF16 gradient

The calls run on the current stream of their operands' device, or on
``stream`` (a torch stream of that device).  As with ``torch.cuda.stream``,
nothing is ordered: the caller lets ``stream`` wait for whatever made the
operands (``stream.wait_stream(torch.cuda.current_stream())``), and lets other
streams wait for it before they use the results.  Memory is held: operands may
be dropped as soon as the call returns, and results as soon as the work that
uses them is queued on ``stream`` or on the stream that was current at the
call.  For any other stream, ``record_stream`` of the tensors and of
``MXMatrix`` tells the allocator.

The calls are not recorded by autograd: the backward calls are the layer's
backward pass.  A dense operand or result whose gradient would be lost (it
requires one and gradients are recorded, or it carries a forward tangent) is
refused, except by ``quantize``: call under ``torch.no_grad()``, from a
``torch.autograd.Function``, or with ``x.detach()``.
"""
from __future__ import annotations

import struct

import torch
from torch.autograd import forward_ad

from . import api

FORMATS = {"fp4": api.MX_FP4, "fp8": api.MX_FP8}
ACTIVATIONS = {"gelu": api.MX_GELU, "gelu_erf": api.MX_GELU_ERF, "swiglu": api.MX_SWIGLU}
_DTYPES = {torch.float32: api.MX_F32, torch.bfloat16: api.MX_BF16}
_BOTH = tuple(_DTYPES)
_PACK = struct.Struct("@iiqqPP").pack   # a q4mx_matrix


class MXMatrix:
    """rows x cols values in format "fp4" or "fp8".

    codes:  uint8 [rows, P / 2] ("fp4") or [rows, P], P = cols rounded up to
            a multiple of 128;
    scales: uint8 [P / 128, rows, 4].
    """
    __slots__ = ("rows", "cols", "format", "device", "packed", "_codes", "_scales", "_buf")

    def __init__(self, rows: int, cols: int, format: str, codes=None, scales=None, device="cuda"):
        if format not in FORMATS:
            raise ValueError(f"unknown format {format!r}; expected one of {sorted(FORMATS)}")
        code = FORMATS[format]
        padded = (cols + 127) // 128 * 128
        if not (0 <= rows < 1 << 31 and 0 <= cols < 1 << 31 and rows * padded < 1 << 34):
            api.q4mx_matrix_bytes(code, rows, cols)   # refuses them, with the reason
        ncodes, nscales = rows * padded // (2 if code == api.MX_FP4 else 1), rows * padded // 32
        self.rows, self.cols, self.format = rows, cols, format
        self._codes, self._scales, self._buf = codes, scales, None
        if codes is None and scales is None:
            # one buffer for both; the views are made when they are asked for
            offset = (ncodes + 255) // 256 * 256
            self._buf = buf = torch.empty(offset + nscales, dtype=torch.uint8, device=device)
            self.device = buf.device
            if not buf.is_cuda:
                raise ValueError("device must be a GPU")
            at = buf.data_ptr()
            pointers = (at, at + offset)
        elif codes is None or scales is None:
            raise ValueError("codes and scales come together")
        else:
            for name, t, shape in (("codes", codes, self._code_shape()), ("scales", scales, self._scale_shape())):
                if t.dtype != torch.uint8 or tuple(t.shape) != shape or not t.is_contiguous():
                    raise ValueError(f"{name} must be a contiguous uint8 tensor of shape {shape}")
                if not t.is_cuda:
                    raise ValueError(f"{name} must be on a GPU")
            if codes.device != scales.device:
                raise ValueError("codes and scales must be on one device")
            self.device = codes.device
            pointers = (codes.data_ptr(), scales.data_ptr())
        self.packed = _PACK(code, 0, rows, cols, *pointers)   # for the calls

    def __reduce__(self):
        # a copy or a pickled matrix describes its own memory, not this one's
        return MXMatrix, (self.rows, self.cols, self.format, self.codes, self.scales)

    @property
    def desc(self) -> api.Q4MXMatrix:
        """The C description of the matrix."""
        return api.Q4MXMatrix.from_buffer_copy(self.packed)

    def _code_shape(self) -> tuple:
        return (self.rows, (self.cols + 127) // 128 * (64 if self.format == "fp4" else 128))

    def _scale_shape(self) -> tuple:
        return ((self.cols + 127) // 128, self.rows, 4)

    @property
    def codes(self):
        if self._codes is None:
            shape = self._code_shape()
            self._codes = self._buf[:shape[0] * shape[1]].view(shape)
        return self._codes

    @property
    def scales(self):
        if self._scales is None:
            shape = self._scale_shape()
            n = shape[0] * shape[1] * 4
            self._scales = self._buf[self._buf.numel() - n:].view(shape)
        return self._scales

    @property
    def shape(self) -> tuple:
        return (self.rows, self.cols)

    def record_stream(self, stream) -> None:
        """torch.Tensor.record_stream of the codes and scales: their memory,
        once freed, is not used again before the work queued on stream by then
        is done."""
        for t in (self._codes, self._scales) if self._buf is None else (self._buf,):
            t.record_stream(stream)

    def __repr__(self) -> str:
        return f"MXMatrix({self.rows} x {self.cols}, {self.format!r}, device='{self.device}')"


def _lost_gradient(t) -> bool:
    """Whether autograd expects to see what is done with t."""
    if t.requires_grad and torch.is_grad_enabled():
        return True
    return forward_ad._current_level >= 0 and forward_ad.unpack_dual(t).tangent is not None


def _dense(name, t, dtypes=(torch.bfloat16,), recorded=True):
    """A 2-D GPU tensor with consecutive columns; returns its row stride."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, not {t.dtype}")
    if recorded and _lost_gradient(t):
        raise ValueError(f"{name} has a gradient, which autograd would lose here; call under torch.no_grad() or detach it")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU")
    rows, cols = t.shape
    ld, step = t.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{name} must have consecutive columns (stride 1)")
    # the stride of a single row, or of an empty matrix, means nothing
    return ld if rows > 1 and cols > 0 else max(1, cols)


def _matrix(name, m):
    if not isinstance(m, MXMatrix):
        raise ValueError(f"{name} must be an MXMatrix")
    return m


def _result(out, shape, dtype, device):
    """(result, its dtype code, its row stride)."""
    if out is None:
        if dtype not in _DTYPES:
            raise ValueError(f"dtype must be torch.float32 or torch.bfloat16, not {dtype}")
        return torch.empty(shape, dtype=dtype, device=device), _DTYPES[dtype], max(1, shape[1])
    ld = _dense("out", out, _BOTH)
    if tuple(out.shape) != tuple(shape):
        raise ValueError(f"out must have shape {tuple(shape)}, not {tuple(out.shape)}")
    if out.shape[0] > 1 and ld < out.shape[1]:
        raise ValueError("out's rows overlap")
    return out, _DTYPES[out.dtype], ld


def _mx_result(out, rows, cols, fmt, device):
    if out is None:
        return MXMatrix(rows, cols, fmt, device=device)
    if _matrix("out", out).shape != (rows, cols) or out.format != fmt:
        raise ValueError(f"out must be a {rows} x {cols} MXMatrix in {fmt!r}")
    return out


def _same_device(first, *others):
    device = first.device
    for t in others:
        if t is not None and t.device != device:
            raise ValueError(f"the operands are on different devices ({device} and {t.device})")
    return device


def _elsewhere(device, stream) -> bool:
    """Whether a call has to enter its device or stream first."""
    return stream is not None or torch._C._cuda_getDevice() != device.index


def _entered(device, stream, operands, call, *args):
    """call(*args) on `device`, or on `stream`.  The allocator knows the stream
    a tensor was made on; the other one that uses it is recorded."""
    if stream is None:
        with torch.cuda.device(device):
            return call(*args)
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the operands on {device}")
    caller = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):   # makes the stream's device current
        results = call(*args)
    _hold(operands, stream)
    _hold(results, caller)
    return results


def _hold(held, stream):
    if isinstance(held, tuple):
        for h in held:
            _hold(h, stream)
    elif held is not None:
        held.record_stream(stream)


def _raw(device) -> int:
    """The current stream of the operands' device, as the C calls take it."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _workspace(nbytes, device):
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def quantize(src, format: str, transpose: bool = False, out: MXMatrix | None = None, stream=None) -> MXMatrix:
    """src (float32 or bfloat16) in a microscaled format, blocks along its
    columns; transpose: the quantized transpose, blocks along its rows (a
    weight whose master is stored [in, out])."""
    ld = _dense("src", src, _BOTH, recorded=False)   # codes have no gradient; the products' calls give that of src
    if format not in FORMATS:
        raise ValueError(f"unknown format {format!r}; expected one of {sorted(FORMATS)}")
    device = src.device
    if out is not None:
        _same_device(src, out)
    if _elsewhere(device, stream):
        return _entered(device, stream, (src, out), quantize, src, format, transpose, out)
    rows, cols = src.shape[::-1] if transpose else src.shape
    out = _mx_result(out, rows, cols, format, device)
    api.q4mx_quantize(src.data_ptr(), _DTYPES[src.dtype], ld, transpose, out.packed, _raw(device))
    return out


def dequantize(a: MXMatrix, dtype=torch.bfloat16, out=None, stream=None) -> torch.Tensor:
    """The values of a."""
    device = _matrix("a", a).device
    if out is not None:
        _same_device(a, out)
    if _elsewhere(device, stream):
        return _entered(device, stream, (a, out), dequantize, a, dtype, out)
    out, code, ld = _result(out, (a.rows, a.cols), dtype, device)
    api.q4mx_dequantize(a.packed, out.data_ptr(), code, ld, _raw(device))
    return out


def linear(x, w: MXMatrix, out=None, dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """x w^T: x an MXMatrix [tokens, in] or a bfloat16 tensor (quantized to
    "fp8" on the way), w an MXMatrix [out, in] in "fp4"."""
    device = _same_device(x, _matrix("w", w), out)
    coded = isinstance(x, MXMatrix)
    if not coded:
        ldx = _dense("x", x)
        if x.shape[1] != w.cols:
            raise ValueError(f"x has {x.shape[1]} columns, w has {w.cols}")
    if _elsewhere(device, stream):
        return _entered(device, stream, (x, w, out), linear, x, w, out, dtype)
    tokens = x.rows if coded else x.shape[0]
    out, code, ld = _result(out, (tokens, w.rows), dtype, device)
    need = 0
    if tokens > api.MX_FEW_TOKENS:
        need = (api.q4mx_linear_workspace_bytes(x.packed, w.packed) if coded
                else api.q4mx_linear_bf16_workspace_bytes(tokens, w.packed))
    ws = _workspace(need, device)
    if coded:
        api.q4mx_linear(x.packed, w.packed, out.data_ptr(), code, ld, ws, need, _raw(device))
    else:
        api.q4mx_linear_bf16(x.data_ptr(), ldx, tokens, w.packed, out.data_ptr(), code, ld, ws, need, _raw(device))
    return out


def linear_dgrad(dy, w: MXMatrix, out=None, dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """dy w: the gradient of linear's x, dy bfloat16 [tokens, out]."""
    lddy = _dense("dy", dy)
    device = _same_device(dy, _matrix("w", w), out)
    tokens, n = dy.shape
    if n != w.rows:
        raise ValueError(f"dy has {n} columns, w has {w.rows} rows")
    if _elsewhere(device, stream):
        return _entered(device, stream, (dy, w, out), linear_dgrad, dy, w, out, dtype)
    out, code, ld = _result(out, (tokens, w.cols), dtype, device)
    at = dy.data_ptr()
    need = api.q4mx_dgrad_workspace_bytes(at, lddy, tokens, w.packed)
    api.q4mx_dgrad(at, lddy, tokens, w.packed, out.data_ptr(), code, ld, _workspace(need, device), need, _raw(device))
    return out


def linear_wgrad(dy, x: MXMatrix, out=None, transposed: bool = False, accumulate: bool = False,
                 dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """dy^T x [out, in], or with transposed its transpose [in, out], from the
    checkpoint x: the gradient of linear's w.  accumulate: added to out."""
    lddy = _dense("dy", dy)
    device = _same_device(dy, _matrix("x", x), out)
    tokens, n = dy.shape
    if tokens != x.rows:
        raise ValueError(f"dy has {tokens} rows, x has {x.rows}")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    if _elsewhere(device, stream):
        return _entered(device, stream, (dy, x, out), linear_wgrad, dy, x, out, transposed, accumulate, dtype)
    flags = (api.MX_WGRAD_TRANSPOSED if transposed else 0) | (api.MX_WGRAD_ADD if accumulate else 0)
    out, code, ld = _result(out, (x.cols, n) if transposed else (n, x.cols), dtype, device)
    at = dy.data_ptr()
    need = api.q4mx_wgrad_workspace_bytes(at, lddy, n, x.packed, flags)
    api.q4mx_wgrad(at, lddy, n, x.packed, out.data_ptr(), code, ld, flags, _workspace(need, device), need, _raw(device))
    return out


def _activation(kind):
    if kind not in ACTIVATIONS:
        raise ValueError(f"unknown activation {kind!r}; expected one of {sorted(ACTIVATIONS)}")
    return ACTIVATIONS[kind]


def act_forward(kind: str, x, up=None, out_format: str | None = None, stream=None):
    """(y, kept): y = f(x) for "gelu" (tanh form) and "gelu_erf", x / (1 +
    e^-x) * up for "swiglu", as a bfloat16 tensor or, with out_format, as an
    MXMatrix (the next linear layer's operand); kept is what act_backward
    needs, the inputs in 8 bits."""
    act = _activation(kind)
    ldx, ldup, up_at = _dense("x", x), 0, None
    if (up is not None) != (kind == "swiglu"):
        raise ValueError('"swiglu" takes up, the others do not')
    device = x.device
    if up is not None:
        ldup, up_at = _dense("up", up), up.data_ptr()
        if up.shape != x.shape:
            raise ValueError("x and up must have one shape")
        _same_device(x, up)
    if out_format is not None and out_format not in FORMATS:
        raise ValueError(f"unknown format {out_format!r}; expected one of {sorted(FORMATS)}")
    if _elsewhere(device, stream):
        return _entered(device, stream, (x, up), act_forward, kind, x, up, out_format)
    rows, cols = x.shape
    y_at = y_mx = None
    if out_format is None:
        y = torch.empty((rows, cols), dtype=torch.bfloat16, device=device)
        y_at = y.data_ptr()
    else:
        y = MXMatrix(rows, cols, out_format, device=device)
        y_mx = y.packed
    kept_x = MXMatrix(rows, cols, "fp8", device=device)
    kept_up = None if up is None else MXMatrix(rows, cols, "fp8", device=device)
    api.q4mx_act_forward(act, x.data_ptr(), ldx, up_at, ldup, rows, cols, y_at, max(1, cols), y_mx, kept_x.packed,
                         None if up is None else kept_up.packed, _raw(device))
    return y, (kept_x, kept_up)


def act_backward(kind: str, kept, dy, stream=None) -> tuple:
    """(dx,) or, for "swiglu", (dx, dup), from act_forward's kept."""
    act = _activation(kind)
    kept_x, kept_up = kept
    _matrix("kept[0]", kept_x)
    if (kept_up is not None) != (kind == "swiglu"):
        raise ValueError('"swiglu" keeps up, the others do not')
    lddy = _dense("dy", dy)
    shape = (kept_x.rows, kept_x.cols)
    if tuple(dy.shape) != shape:
        raise ValueError(f"dy must have shape {shape}, not {tuple(dy.shape)}")
    device = _same_device(dy, kept_x, kept_up)
    if _elsewhere(device, stream):
        return _entered(device, stream, (kept_x, kept_up, dy), act_backward, kind, kept, dy)
    ld = max(1, shape[1])
    dx = torch.empty(shape, dtype=torch.bfloat16, device=device)
    dup = None if kept_up is None else torch.empty(shape, dtype=torch.bfloat16, device=device)
    api.q4mx_act_backward(act, kept_x.packed, None if dup is None else kept_up.packed, dy.data_ptr(), lddy,
                          dx.data_ptr(), ld, None if dup is None else dup.data_ptr(), ld, _raw(device))
    return (dx,) if dup is None else (dx, dup)
