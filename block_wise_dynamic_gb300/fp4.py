"""Linear layers on microscaled 4-bit floating point operands (e2m1 codes, a
power-of-two scale for each block of 32 along a row, sm_103a).

A block's scale is 2^e with the smallest e >= -127 for which no magnitude in
it exceeds 6 * 2^e; codes are rounded to nearest, ties to even.  For serving
what was trained at more bits: a weight takes 17/32 of a byte an element.  A
matrix that is quantized, or read back, has at most 2,097,120 rows.

  quantize(x) -> Fp4Matrix          blocks of 1 x 32 along the rows
  dequantize(q)                     the values that the codes stand for
  matmul(a, b, bias)                A B^T of two quantized matrices
  linear(x, w, bias)                the product with a weight kept quantized
  Fp4Linear                         torch.nn.Module around it, for inference

Each function checks and marshals CUDA tensors and calls ``bwd_fp4_*`` of
``include/bwd.h``; quantization and products run in the library's kernels.
"""

from __future__ import annotations

from functools import lru_cache
from typing import Optional

import torch

from . import _GDT, _launch, _need
from ._once import has_tangent
from .fp8 import _bytes, _matrix, _on, _ptr, _round256

__all__ = ["Fp4Matrix", "quantize", "dequantize", "matmul", "linear", "Fp4Linear"]


@lru_cache(maxsize=1024)
def _layout(rows: int, cols: int):
    """Bytes between rows of codes, where the scales begin, and where they
    end: bwd_fp4_pitch and bwd_fp4_scale_bytes."""
    row = (cols + 1) // 2
    pitch = (row + 127) // 128 * 128 if row > 64 else (row + 15) // 16 * 16
    codes = _round256(rows * pitch)
    return pitch, codes, codes + (rows + 127) // 128 * ((cols + 255) // 256) * 1024


class Fp4Matrix:
    """A rows x cols matrix in e2m1 codes, two to a byte (``codes``, a row's
    bytes up to its pitch), and the scales' bytes in tiles (``scales``); both
    lie in ``buffer``."""

    __slots__ = ("shape", "dtype", "device", "buffer", "_pointers")

    def __init__(self, rows: int, cols: int, dtype, buffer: torch.Tensor):
        """Over a buffer that was another such matrix's, or will be filled."""
        _need(buffer, "buffer", torch.uint8, _layout(rows, cols)[2])
        if dtype not in _GDT:
            raise TypeError("dtype must be float32, bfloat16 or float16")
        self._place(rows, cols, dtype, buffer if buffer.data_ptr() % 16 == 0 else buffer.clone(), buffer.device)

    def _place(self, rows, cols, dtype, buffer, device):
        self.shape, self.dtype, self.device, self.buffer = (rows, cols), dtype, device, buffer
        base = buffer.data_ptr()
        self._pointers = base, base + _layout(rows, cols)[1]  # addresses of codes and scales

    @property
    def codes(self) -> torch.Tensor:
        pitch = _layout(*self.shape)[0]
        return self.buffer[:self.shape[0] * pitch].view(self.shape[0], pitch)

    @property
    def scales(self) -> torch.Tensor:
        return self.buffer[_layout(*self.shape)[1]:]

    def dequantize(self, dtype=None, stream=None) -> torch.Tensor:
        return dequantize(self, dtype, stream)


def _fp4(a, name):
    if not isinstance(a, Fp4Matrix):
        raise TypeError(f"{name} must be an Fp4Matrix")
    return a


def quantize(x: torch.Tensor, stream=None) -> Fp4Matrix:
    """Quantizes a matrix (leading dimensions are flattened) in blocks of 1 x 32."""
    if stream is not None:
        with _on(stream, x.device):
            return quantize(x)
    x = _matrix(x, "x")
    rows, cols = x.shape
    dev, dtype = x.device, x.dtype
    q = Fp4Matrix.__new__(Fp4Matrix)
    q._place(rows, cols, dtype, _bytes(_layout(rows, cols)[2], dev), dev)
    _launch("bwd_fp4_quantize", dev, None, x.data_ptr(), _GDT[dtype], rows, cols, max(x.stride(0), cols), *q._pointers)
    return q


def dequantize(a: Fp4Matrix, dtype=None, stream=None) -> torch.Tensor:
    """The values that the codes stand for, in ``dtype`` (the quantized tensor's by default)."""
    _fp4(a, "a")
    if stream is not None:
        with _on(stream, a.device):
            return dequantize(a, dtype)
    dtype = a.dtype if dtype is None else dtype
    if dtype not in _GDT:
        raise TypeError("dtype must be float32, bfloat16 or float16")
    out = torch.empty(a.shape, dtype=dtype, device=a.device)
    _launch("bwd_fp4_dequantize", a.device, None, *a._pointers, *a.shape, out.data_ptr(), _GDT[dtype])
    return out


def matmul(a: Fp4Matrix, b: Fp4Matrix, bias: Optional[torch.Tensor] = None, dtype=None, stream=None) -> torch.Tensor:
    """A B^T plus a row of biases, in ``dtype`` (the type that a was quantized from by default)."""
    m, k = _fp4(a, "a").shape
    n, kb = _fp4(b, "b").shape
    if k != kb:
        raise ValueError(f"a's rows have {k} elements, b's {kb}")
    if b.device != a.device:
        raise ValueError(f"b is on {b.device}, the call runs on {a.device}")
    if stream is not None:
        with _on(stream, a.device):
            return matmul(a, b, bias, dtype)
    dtype = a.dtype if dtype is None else dtype
    if dtype not in _GDT:
        raise TypeError("dtype must be float32, bfloat16 or float16")
    if bias is not None:
        _need(bias, "bias", dtype, n, a.device)
    out = torch.empty((m, n), dtype=dtype, device=a.device)
    _launch("bwd_fp4_matmul", a.device, None, m, n, k, *a._pointers, *b._pointers, _ptr(bias), out.data_ptr(), n, _GDT[dtype])
    return out


_FUSED_ROWS, _FUSED_COLS = 8, 229_376  # what the library's product quantizes itself, without a workspace


@lru_cache(maxsize=1024)
def _work(rows: int, cols: int) -> int:
    """bwd_fp4_linear_work_bytes."""
    if rows <= _FUSED_ROWS and cols <= _FUSED_COLS:
        return 0
    return _round256(_layout(rows, cols)[2])


def linear(x: torch.Tensor, w: Fp4Matrix, bias: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """x W^T + bias in x's dtype, for a quantized weight (outputs x inputs); x
    is quantized within the call.  No gradients."""
    n, width = _fp4(w, "w").shape
    if stream is not None:
        with _on(stream, x.device):
            return linear(x, w, bias)
    m = _matrix(x, "x")
    rows, cols = m.shape
    dev = m.device
    if cols != width:
        raise ValueError(f"x's last dimension must be {width}")
    if w.device != dev:
        raise ValueError(f"w is on {w.device}, the call runs on {dev}")
    if bias is not None:
        _need(bias, "bias", m.dtype, n, dev)
    y = torch.empty((rows, n) if m is x else (*x.shape[:-1], n), dtype=m.dtype, device=dev)
    size = _work(rows, cols)
    work = _bytes(size, dev) if size else None
    _launch("bwd_fp4_linear", dev, None, m.data_ptr(), _GDT[m.dtype], rows, cols, max(m.stride(0), cols), *w._pointers, n, _ptr(bias),
            y.data_ptr(), n, _ptr(work))
    return y


class Fp4Linear(torch.nn.Module):
    """Linear layer for inference on a weight kept in 4 bits, made from a
    trained layer (``torch.nn.Linear``, :class:`.fp8.Fp8Linear` or any with
    ``weight`` and ``bias``).  ``quantized`` is a buffer: it is saved with the
    module and moves between devices with it."""

    def __init__(self, layer: torch.nn.Module):
        super().__init__()
        weight = layer.weight.detach()
        if weight.dim() != 2:
            raise ValueError("the layer's weight must be a matrix")
        q = quantize(weight)
        self.out_features, self.in_features = q.shape
        self.dtype = q.dtype
        self.register_buffer("quantized", q.buffer)
        bias = getattr(layer, "bias", None)
        self.register_buffer("bias", None if bias is None else bias.detach().clone())

    @property
    def weight(self) -> Fp4Matrix:
        return Fp4Matrix(self.out_features, self.in_features, self.dtype, self.quantized)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if has_tangent(x) or torch.is_grad_enabled() and x.requires_grad:
            raise RuntimeError("Fp4Linear has no gradients: use it under torch.no_grad()")
        bias = self.bias if self.bias is None or self.bias.dtype == x.dtype else self.bias.to(x.dtype)
        return linear(x, self.weight, bias)
