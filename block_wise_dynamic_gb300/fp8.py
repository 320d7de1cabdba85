"""Linear layers on 8-bit floating point operands with a power-of-two scale
for each block of 128 (e4m3 codes, sm_103a).

A block's scale is 2^e with the smallest e >= -127 for which no magnitude in
it exceeds 448 * 2^e; codes are rounded to nearest, ties to even.  Each of a
layer's three products sums over blocks of its own operands:

  y  = Q(x) Q(w)^T + bias   x in blocks of 1 x 128, w of 128 x 128
  dx = Q(dy) Q(w)           dy in blocks of 1 x 128
  dw = Q(dy)^T Q(x)         dy and x in blocks of 128 x 1

  quantize(x, "rows" | "cols" | "both" | "tiles") -> Fp8Matrix
  matmul(a, b, trans_a, trans_b, bias)            A B^T of two quantized matrices
  linear(x, w, bias)                              the product with a weight kept quantized
  forward(x, w, bias) -> (y, xq);  backward(dy, xq, w) -> (dx, dw, dbias)
  Fp8Linear                                       torch.nn.Module with autograd through them

Each function checks and marshals CUDA tensors and calls ``bwd_fp8_*`` of
``include/bwd.h``; quantization and products run in the library's kernels.
"""

from __future__ import annotations

from functools import lru_cache
from typing import Optional

import torch

from . import _abi
from . import _GDT, _launch, _need
from ._once import first_order

__all__ = ["Fp8Matrix", "quantize", "dequantize", "matmul", "linear", "forward", "backward", "Fp8Linear"]

_BLOCKS = {"rows": _abi.FP8_ROWS, "cols": _abi.FP8_COLS, "both": _abi.FP8_ROWS | _abi.FP8_COLS, "tiles": _abi.FP8_TILES}
_FUSED_ROWS, _FUSED_COLS = 16, 245_760  # what the library's product quantizes itself, without a workspace
# Up to this many bytes of workspace lie behind the matrix that forward() returns
# and live as long: such calls take less time than an allocation costs (2.5 of
# some 58 us for a training pass of 300 x 704 x 304).
_ROOM = 1 << 20


class Fp8Matrix:
    """A rows x cols matrix in e4m3 codes.  ``row_codes`` / ``row_scales`` are
    quantized in blocks along the rows, ``col_codes`` / ``col_scales`` along
    the columns (None where ``blocks`` has no such form); with "tiles" both
    are the same codes.  All lie in one buffer."""

    __slots__ = ("shape", "blocks", "dtype", "device", "buffer", "_places", "_pointers")

    def __init__(self, rows: int, cols: int, blocks: str, dtype, device, room: int = 0):
        """``room``: bytes that the buffer has beyond the matrix, from a multiple of 256 on."""
        end = _layout(rows, cols, _BLOCKS[blocks])[4]
        self._place(rows, cols, blocks, dtype, _bytes(_round256(end) + room if room else end, device))

    def _place(self, rows, cols, blocks, dtype, buffer):
        self.shape, self.blocks, self.dtype, self.device, self.buffer = (rows, cols), blocks, dtype, buffer.device, buffer
        rc, rs, cc, cs, _ = self._places = _layout(rows, cols, _BLOCKS[blocks])
        # addresses of row codes, row scales, column codes, column scales
        base = self.buffer.data_ptr()
        self._pointers = (None if rc is None else base + rc, None if rs is None else base + rs,
                          None if cc is None else base + cc, None if cs is None else base + cs)

    @classmethod
    def _over(cls, like, buffer: torch.Tensor):
        """The matrix whose ``_like()`` that was, in a buffer with the same bytes."""
        if not buffer.is_contiguous() or buffer.data_ptr() % 16:
            buffer = buffer.clone(memory_format=torch.contiguous_format)
        q = cls.__new__(cls)
        q._place(*like, buffer)
        return q

    def _like(self):
        return (*self.shape, self.blocks, self.dtype)

    def _view(self, which, size):
        at = self._places[which]
        return None if at is None else self.buffer[at:at + size]

    def _codes(self, which):
        rows, cols = self.shape
        v = self._view(which, rows * _pitch(cols))
        return None if v is None else v.view(rows, _pitch(cols))

    @property
    def row_codes(self):
        return self._codes(0)

    @property
    def row_scales(self):
        return self._view(1, _scale_bytes(*self.shape))

    @property
    def col_codes(self):
        return self._codes(2)

    @property
    def col_scales(self):
        return self._view(3, _scale_bytes(self.shape[1], self.shape[0]))

    def dequantize(self, along="rows", dtype=None, stream=None):
        return dequantize(self, along, dtype, stream)


@lru_cache(maxsize=1024)
def _layout(rows: int, cols: int, kind: int):
    """Offsets in a matrix's buffer of row codes, row scales, column codes and
    column scales, and the buffer's size."""
    codes = _round256(rows * _pitch(cols))
    rc = rs = cc = cs = None
    end = 0
    if kind & (_abi.FP8_ROWS | _abi.FP8_TILES):
        rc, rs = 0, codes
        end = codes + _round256(_scale_bytes(rows, cols))
    if kind & _abi.FP8_COLS:
        cc, cs = end, end + codes
        end += codes + _scale_bytes(cols, rows)
    elif kind & _abi.FP8_TILES:
        cc, cs = 0, end
        end += _scale_bytes(cols, rows)
    return rc, rs, cc, cs, end


@lru_cache(maxsize=1024)
def _forward_work(rows: int, cols: int) -> int:
    """bwd_fp8_linear_work_bytes."""
    if rows <= _FUSED_ROWS and cols <= _FUSED_COLS:
        return 0
    return _round256(rows * _pitch(cols)) + _round256(_scale_bytes(rows, cols))


@lru_cache(maxsize=1024)
def _backward_work(rows: int, n: int) -> int:
    """bwd_fp8_linear_backward_work_bytes."""
    return (2 * _round256(rows * _pitch(n)) + _round256(_scale_bytes(rows, n)) + _round256(_scale_bytes(n, rows)) +
            _round256((rows + 127) // 128 * n * 4))


def _pitch(cols: int) -> int:
    return (cols + 127) // 128 * 128 if cols > 64 else (cols + 15) // 16 * 16


def _scale_bytes(count: int, length: int) -> int:
    return (count + 127) // 128 * ((length + 511) // 512) * 512


def _round256(n: int) -> int:
    return (n + 255) // 256 * 256


def _matrix(x: torch.Tensor, name: str) -> torch.Tensor:
    """x as a 2-d matrix with contiguous rows."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if x.dtype not in _GDT:
        raise TypeError(f"{name} must be float32, bfloat16 or float16")
    if x.dim() != 2:
        if x.dim() == 0:
            raise ValueError(f"{name} must have at least one dimension")
        x = x.reshape(x.shape[:-1].numel(), x.shape[-1])
    if not x.is_contiguous() and (x.stride(1) != 1 or x.stride(0) < x.shape[1]):
        x = x.contiguous()
    return x


def _on(stream, device):
    """Context in which ``stream`` (a torch stream or a handle) is current: a
    call's temporaries, copies and results belong to the stream they are used
    on."""
    return torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(stream, device))


def _bytes(n: int, device: torch.device) -> torch.Tensor:
    return torch.empty(n, dtype=torch.uint8, device=device)


def _ptr(t):
    return None if t is None else t.data_ptr()


def quantize(x: torch.Tensor, blocks: str = "rows", col_sums: bool = False, stream=None):
    """Quantizes a matrix (leading dimensions are flattened).  With
    ``col_sums`` (for "cols" and "both") returns (matrix, sums of the columns
    in x's dtype)."""
    if blocks not in _BLOCKS:
        raise ValueError(f"blocks must be one of {sorted(_BLOCKS)}")
    kind = _BLOCKS[blocks]
    if col_sums and not kind & _abi.FP8_COLS:
        raise ValueError('column sums need blocks "cols" or "both"')
    if stream is not None:
        with _on(stream, x.device):
            return quantize(x, blocks, col_sums)
    x = _matrix(x, "x")
    rows, cols = x.shape
    dev = x.device
    q = Fp8Matrix(rows, cols, blocks, x.dtype, dev)
    rc, rs, cc, cs = q._pointers
    sums = work = None
    if col_sums:
        sums = torch.empty(cols, dtype=x.dtype, device=dev)
        work = torch.empty(max(1, (rows + 127) // 128 * cols), dtype=torch.float32, device=dev)
    _launch("bwd_fp8_quantize", dev, None, x.data_ptr(), _GDT[x.dtype], rows, cols, max(x.stride(0), cols), kind, rc, rs, cc, cs,
            _ptr(sums), _ptr(work))
    return (q, sums) if col_sums else q


def _lines(a: Fp8Matrix, trans: bool, name: str):
    """Addresses of codes and scales, number and length of a matrix's lines."""
    if not isinstance(a, Fp8Matrix):
        raise TypeError(f"{name} must be an Fp8Matrix")
    rows, cols = a.shape
    codes, scales = a._pointers[2:] if trans else a._pointers[:2]
    if codes is None:
        raise ValueError(f'{name} has blocks "{a.blocks}", the product sums along its {"columns" if trans else "rows"}')
    return (codes, scales, cols, rows) if trans else (codes, scales, rows, cols)


def dequantize(a: Fp8Matrix, along: str = "rows", dtype=None, stream=None) -> torch.Tensor:
    """The values that the codes stand for, in ``dtype`` (the quantized
    tensor's by default); ``along`` picks the row or the column form."""
    if along not in ("rows", "cols"):
        raise ValueError('along must be "rows" or "cols"')
    codes, scales, _, _ = _lines(a, along == "cols", "a")
    if stream is not None:
        with _on(stream, a.device):
            return dequantize(a, along, dtype)
    dtype = a.dtype if dtype is None else dtype
    if dtype not in _GDT:
        raise TypeError("dtype must be float32, bfloat16 or float16")
    rows, cols = a.shape
    out = torch.empty((rows, cols), dtype=dtype, device=a.device)
    _launch("bwd_fp8_dequantize", a.device, None, codes, scales, int(along == "rows"), rows, cols, out.data_ptr(), _GDT[dtype])
    return out


def matmul(a: Fp8Matrix, b: Fp8Matrix, trans_a: bool = False, trans_b: bool = False, bias: Optional[torch.Tensor] = None,
           dtype=None, stream=None) -> torch.Tensor:
    """out[i, j] = sum over the lines' elements of A's line i and B's line j,
    plus bias[j].  A matrix's lines are its rows, or with ``trans`` its
    columns; the blocks must run along them."""
    ac, asc, m, k = _lines(a, trans_a, "a")
    bc, bsc, n, kb = _lines(b, trans_b, "b")
    if k != kb:
        raise ValueError(f"a's lines have {k} elements, b's {kb}")
    if stream is not None:
        with _on(stream, a.device):
            return matmul(a, b, trans_a, trans_b, bias, dtype)
    dev = a.device
    if b.device != dev:
        raise ValueError(f"b is on {b.device}, the call runs on {dev}")
    dtype = a.dtype if dtype is None else dtype
    if dtype not in _GDT:
        raise TypeError("dtype must be float32, bfloat16 or float16")
    if bias is not None:
        _need(bias, "bias", dtype, n, dev)
    out = torch.empty((m, n), dtype=dtype, device=dev)
    _launch("bwd_fp8_matmul", dev, None, m, n, k, ac, int(trans_a), asc, bc, int(trans_b), bsc, _ptr(bias), out.data_ptr(), n,
            _GDT[dtype])
    return out


def _operands(x: torch.Tensor, w: Fp8Matrix, axis: int, name: str):
    """x as a matrix whose width is w's ``axis``, and the addresses of w's codes
    and scales for lines along it (the row form for axis 1, the column form
    for axis 0)."""
    m = _matrix(x, name)
    codes, scales, _, width = _lines(w, axis == 0, "w")
    if m.shape[1] != width:
        raise ValueError(f"{name}'s last dimension must be {width}")
    if w.device != m.device:
        raise ValueError(f"w is on {w.device}, the call runs on {m.device}")
    return m, codes, scales


def _forward(x, w, bias, both, stream):
    if stream is not None:
        with _on(stream, x.device):
            return _forward(x, w, bias, both, None)
    m, codes, scales = _operands(x, w, 1, "x")
    rows, cols = m.shape
    n, dev, dt = w.shape[0], m.device, m.dtype
    if bias is not None:
        _need(bias, "bias", dt, n, dev)
    y = torch.empty((rows, n) if m is x else (*x.shape[:-1], n), dtype=dt, device=dev)
    work = cc = cs = xq = None
    size = _forward_work(rows, cols)
    if both:
        room = size if size <= _ROOM else 0
        xq = Fp8Matrix(rows, cols, "cols", dt, dev, room)
        _, _, cc, cs = xq._pointers
        if room:
            work = xq.buffer.data_ptr() + xq.buffer.numel() - room
    if size and work is None:
        scratch = _bytes(size, dev)
        work = scratch.data_ptr()
    _launch("bwd_fp8_linear", dev, None, m.data_ptr(), _GDT[dt], rows, cols, max(m.stride(0), cols), codes, scales, n, _ptr(bias),
            y.data_ptr(), n, cc, cs, work)
    return y, xq


def linear(x: torch.Tensor, w: Fp8Matrix, bias: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """x W^T + bias in x's dtype, for a weight (outputs x inputs) quantized
    with blocks "tiles" or "rows"; x is quantized within the call."""
    return _forward(x, w, bias, False, stream)[0]


def forward(x: torch.Tensor, w: Fp8Matrix, bias: Optional[torch.Tensor] = None, stream=None):
    """(y, xq): :func:`linear`, and x quantized in column blocks, which
    :func:`backward` reads."""
    return _forward(x, w, bias, True, stream)


def backward(dy: torch.Tensor, xq: Fp8Matrix, w: Fp8Matrix, need_input: bool = True, need_weight: bool = True,
             need_bias: bool = False, stream=None):
    """(dx, dw, dbias) in dy's dtype, None for those not needed.  xq has
    column blocks (from :func:`forward`), w blocks "tiles" or "cols"."""
    if stream is not None:
        with _on(stream, dy.device):
            return backward(dy, xq, w, need_input, need_weight, need_bias)
    m, codes, scales = _operands(dy, w, 0, "dy")
    rows, n = m.shape
    k, dev, dt = w.shape[1], m.device, m.dtype
    xc = xs = dx = dw = db = None
    if need_weight:
        if not isinstance(xq, Fp8Matrix) or tuple(xq.shape) != (rows, k):
            raise ValueError(f"xq must be an Fp8Matrix of shape {(rows, k)}")
        xc, xs, _, _ = _lines(xq, True, "xq")
        if xq.device != dev:
            raise ValueError(f"xq is on {xq.device}, the call runs on {dev}")
        dw = torch.empty((n, k), dtype=dt, device=dev)
    if need_input:
        dx = torch.empty((rows, k) if m is dy else (*dy.shape[:-1], k), dtype=dt, device=dev)
    if need_bias:
        db = torch.empty(n, dtype=dt, device=dev)
    work = _bytes(_backward_work(rows, n), dev)
    _launch("bwd_fp8_linear_backward", dev, None, m.data_ptr(), _GDT[dt], rows, n, max(m.stride(0), n), codes, scales, xc, xs, k,
            _ptr(dx), k, _ptr(dw), k, _ptr(db), work.data_ptr())
    return dx, dw, db


class _Fp8LinearFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, wq):
        # x's column form is read for the weight's gradient alone
        y, xq = forward(x, wq, bias) if ctx.needs_input_grad[1] else (linear(x, wq, bias), None)
        ctx.save_for_backward(wq.buffer, None if xq is None else xq.buffer)
        ctx.like = wq._like(), None if xq is None else xq._like()
        return y

    @staticmethod
    @first_order("Fp8Linear")
    def backward(ctx, dy):
        wq, xq = (None if t is None else Fp8Matrix._over(like, t) for like, t in zip(ctx.like, ctx.saved_tensors))
        dx, dw, db = backward(dy, xq, wq, *ctx.needs_input_grad[:3])
        return dx, dw, db, None


class Fp8Linear(torch.nn.Module):
    """Linear layer whose three products take 8-bit operands.  ``weight``
    (outputs x inputs, Xavier-uniform) and ``bias`` (zeros) are ordinary
    parameters of ``dtype`` for any optimizer; each call quantizes the weight
    as it is then.  It has first derivatives only: differentiating through
    gradients made with ``create_graph`` raises.  :func:`linear` takes a weight quantized once."""

    def __init__(self, in_features: int, out_features: int, bias: bool = True, device=None, dtype=torch.bfloat16):
        super().__init__()
        device = torch.device(device if device is not None else "cuda")
        self.in_features, self.out_features = int(in_features), int(out_features)
        self.weight = torch.nn.Parameter(torch.empty(out_features, in_features, dtype=dtype, device=device))
        self.bias = torch.nn.Parameter(torch.zeros(out_features, dtype=dtype, device=device)) if bias else None
        bound = (6.0 / (in_features + out_features)) ** 0.5
        with torch.no_grad():
            self.weight.uniform_(-bound, bound)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        wq = quantize(self.weight.detach(), "tiles")
        if not torch.is_grad_enabled():
            return linear(x, wq, self.bias)
        return _Fp8LinearFn.apply(x, self.weight, self.bias, wq)
