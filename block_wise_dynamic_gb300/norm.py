"""Layer normalisation over a tensor's last dimension, forward and backward.

  y = (x - mean) / sqrt(var + eps) * gamma + beta      var biased, per row

The stable embedding layer (:mod:`.embedding`) normalises right behind its
lookup; this is the normalisation by itself, for the layers behind it.

  forward(x, gamma, beta, eps) -> (y, mean, rstd)
  backward(dy, x, gamma, mean, rstd) -> (dx, dgamma, dbeta)
  LayerNorm                     torch.nn.Module with autograd through them

x is float32, bfloat16 or float16, gamma and beta float32 or of x's type;
statistics and sums are held in 32 bits.  Each function checks and marshals
CUDA tensors and makes one call into ``libbwd.so`` (``bwd_norm_*`` in
``include/bwd.h``).
"""

from __future__ import annotations

from functools import lru_cache
from typing import Optional

import torch

from . import _abi
from . import _GDT, _launch, _need
from ._once import first_order, without_autograd
from .fp8 import _matrix, _on, _ptr

EPS = 1e-5
MAX_WIDTH = 16384  # elements of a row

__all__ = ["EPS", "MAX_WIDTH", "forward", "backward", "LayerNorm"]


@lru_cache(maxsize=1024)
def _work(rows: int, width: int) -> int:
    return _abi.load().bwd_norm_backward_work_bytes(rows, width) // 4


def _vectors(gamma, beta, x_dtype, width, device):
    """The type of gamma and beta (float32 where there is neither)."""
    one = beta if gamma is None else gamma
    if one is None:
        return torch.float32
    dtype = one.dtype if isinstance(one, torch.Tensor) else None
    if dtype is not torch.float32 and dtype is not x_dtype:
        raise TypeError("gamma and beta must be float32 or of x's dtype")
    if gamma is not None:
        _need(gamma, "gamma", dtype, width, device)
    if beta is not None:
        _need(beta, "beta", dtype, width, device)
    return dtype


def forward(x: torch.Tensor, gamma: Optional[torch.Tensor] = None, beta: Optional[torch.Tensor] = None, eps: float = EPS,
            need_stats: bool = True, stream=None):
    """(y, mean, rstd): y in x's dtype and shape, and float32 statistics of
    each row (None when ``need_stats`` is false).  Without gamma it is 1,
    without beta 0."""
    if stream is not None:
        with _on(stream, x.device):
            return forward(x, gamma, beta, eps, need_stats)
    m = _matrix(x, "x")
    rows, width = m.shape
    if not 1 <= width <= MAX_WIDTH:
        raise ValueError(f"the last dimension must be 1 to {MAX_WIDTH}")
    dev, dtype = m.device, m.dtype
    vectors = _vectors(gamma, beta, dtype, width, dev)
    y = torch.empty((rows, width) if m is x else x.shape, dtype=dtype, device=dev)
    mean = torch.empty(rows, dtype=torch.float32, device=dev) if need_stats else None
    rstd = torch.empty(rows, dtype=torch.float32, device=dev) if need_stats else None
    _launch("bwd_norm_forward", dev, None, m.data_ptr(), _GDT[dtype], rows, width, max(m.stride(0), width), _ptr(gamma), _ptr(beta),
            _GDT[vectors], eps, y.data_ptr(), _ptr(mean), _ptr(rstd))
    return y, mean, rstd


def backward(dy: torch.Tensor, x: torch.Tensor, gamma: Optional[torch.Tensor], mean: torch.Tensor, rstd: torch.Tensor,
             need_input: bool = True, need_gamma: bool = True, need_beta: bool = True, vector_dtype=None, stream=None):
    """(dx, dgamma, dbeta), None for those not needed; dx in x's dtype, the
    others in gamma's (``vector_dtype``, or float32, where there is none)."""
    if stream is not None:
        with _on(stream, x.device):
            return backward(dy, x, gamma, mean, rstd, need_input, need_gamma, need_beta, vector_dtype)
    m, d = _matrix(x, "x"), _matrix(dy, "dy")
    rows, width = m.shape
    if not 1 <= width <= MAX_WIDTH:
        raise ValueError(f"the last dimension must be 1 to {MAX_WIDTH}")
    dev, dtype = m.device, m.dtype
    if dy.shape != x.shape or d.dtype is not dtype:
        raise ValueError(f"dy must have x's shape and dtype, {tuple(x.shape)} {x.dtype}")
    if d.device != dev:
        raise ValueError(f"dy is on {d.device}, the call runs on {dev}")
    vectors = _vectors(gamma, None, dtype, width, dev)
    if gamma is None and vector_dtype is not None:
        vectors = vector_dtype
        if vectors not in (torch.float32, dtype):
            raise TypeError("vector_dtype must be float32 or x's dtype")
    _need(mean, "mean", torch.float32, rows, dev)
    _need(rstd, "rstd", torch.float32, rows, dev)
    dx = torch.empty((rows, width) if m is x else x.shape, dtype=dtype, device=dev) if need_input else None
    dgamma = torch.empty(width, dtype=vectors, device=dev) if need_gamma else None
    dbeta = torch.empty(width, dtype=vectors, device=dev) if need_beta else None
    work = torch.empty(_work(rows, width), dtype=torch.float32, device=dev) if need_gamma or need_beta else None
    _launch("bwd_norm_backward", dev, None, d.data_ptr(), m.data_ptr(), _GDT[dtype], rows, width, max(d.stride(0), width),
            max(m.stride(0), width), _ptr(gamma), _GDT[vectors], mean.data_ptr(), rstd.data_ptr(), _ptr(dx), _ptr(dgamma), _ptr(dbeta),
            _ptr(work))
    return dx, dgamma, dbeta


class _LayerNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gamma, beta, eps):
        y, mean, rstd = forward(x, gamma, beta, eps)
        ctx.save_for_backward(x, gamma, mean, rstd)
        return y

    @staticmethod
    @first_order("LayerNorm")
    def backward(ctx, dy):
        x, gamma, mean, rstd = ctx.saved_tensors
        dx, dgamma, dbeta = backward(dy, x, gamma, mean, rstd, *ctx.needs_input_grad[:3])
        return dx, dgamma, dbeta, None


class LayerNorm(torch.nn.Module):
    """Layer normalisation over the last dimension of ``dim`` elements.
    ``weight`` (ones) and, with ``bias``, ``bias`` (zeros) are float32 unless
    ``dtype`` says otherwise, for activations of any of the types.  It has
    first derivatives in backward mode only: differentiating through gradients
    made with ``create_graph`` raises, and so do inputs with a forward-mode
    tangent."""

    def __init__(self, dim: int, eps: float = EPS, bias: bool = True, device=None, dtype=torch.float32):
        super().__init__()
        device = torch.device(device if device is not None else "cuda")
        self.dim, self.eps = int(dim), float(eps)
        if not 1 <= self.dim <= MAX_WIDTH:
            raise ValueError(f"dim must be 1 to {MAX_WIDTH}")
        self.weight = torch.nn.Parameter(torch.ones(dim, dtype=dtype, device=device))
        self.bias = torch.nn.Parameter(torch.zeros(dim, dtype=dtype, device=device)) if bias else None

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if without_autograd():
            return forward(x, self.weight, self.bias, self.eps, need_stats=False)[0]
        return _LayerNormFn.apply(x, self.weight, self.bias, self.eps)
