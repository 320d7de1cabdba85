"""AdamW with both moments in fp32, and the gradients' norm and clipping factor.

For the tensors of a run whose moments stay in 32 bits beside the 8-bit ones
(an embedding, norms, biases).  Each call checks and marshals CUDA tensors and
makes one call into ``libbwd.so`` (``bwd_adam32_step_multi``, ``bwd_grad_norm``
in ``include/bwd.h``).

    args = MultiTensorArgs32(params, grads, m, v)     # pointer table, built once
    norm = GradNorm(grads)
    factor, _ = norm.clip_scale(1.0)                  # on the device, no synchronisation
    args.step(lr=1e-3, step=t, grad_scale=factor)
"""

from __future__ import annotations

import ctypes
from typing import Sequence

import torch

from . import _abi
from . import _GDT, _launch, _lib, _need

__all__ = ["StepCount", "MultiTensorArgs32", "adam32_step_multi", "GradNorm", "clip_scale"]


def _one_dtype(tensors, what):
    kinds = {t.dtype for t in tensors}
    if len(kinds) > 1:
        raise TypeError(f"all {what} of one call must share a dtype")
    for k in kinds:
        if k not in _GDT:
            raise TypeError(f"{what} must be float32, bfloat16 or float16")
    return _GDT[kinds.pop()] if kinds else _abi.BWD_F32


def _pointers(tensors):
    return (ctypes.c_void_p * len(tensors))(*[t.data_ptr() for t in tensors])


def _check_scale(grad_scale, device):
    if grad_scale is None:
        return None
    _need(grad_scale, "grad_scale", torch.float32, 1, device)
    return grad_scale.data_ptr()


class StepCount:
    """A number of steps taken, held on the device: steps whose factor is not
    finite write nothing and are not counted, which the host does not know.
    ``taken`` is an int64 CUDA tensor of no dimension, the number itself."""

    def __init__(self, device, taken: int = 0):
        self.buffer = torch.full((2,), int(taken), dtype=torch.int64, device=device)
        self.taken = self.buffer[0]


def _count_on(count: StepCount, device) -> int:
    if count.buffer.device != device:
        raise ValueError(f"the step count is on {count.buffer.device}, the call runs on {device}")
    return count.buffer.data_ptr()


class _GradList:
    """Host pointer table of a fixed list of gradients."""

    def _init_grads(self, grads, device):
        self.T = len(grads)
        self.device = device
        for i, g in enumerate(grads):
            _need(g, f"grads[{i}]", g.dtype, None, device)
            if g.dtype not in _GDT:
                raise TypeError("gradients must be float32, bfloat16 or float16")
        self._grads = list(grads)
        self._dtypes = [g.dtype for g in grads]
        self.g = _pointers(grads)
        self._sizes = [g.numel() for g in grads]
        self.n = (ctypes.c_int64 * self.T)(*self._sizes)

    def set_grads(self, grads: Sequence[torch.Tensor]) -> None:
        """Points the table at new gradient tensors of the same sizes, dtypes
        and device (non-contiguous ones are copied)."""
        if len(grads) != self.T:
            raise ValueError(f"expected {self.T} gradients, got {len(grads)}")
        dev = self.device
        if not all(isinstance(g, torch.Tensor) for g in grads) or [g.dtype for g in grads] != self._dtypes:
            raise TypeError("every gradient must be a tensor of the dtype that the table was built for")
        if [g.numel() for g in grads] != self._sizes:
            raise ValueError("gradient sizes differ from those the table was built for")
        if not all(g.device == dev for g in grads):
            raise ValueError(f"every gradient must be on {dev}")
        grads = [g if g.is_contiguous() else g.contiguous() for g in grads]
        self._grads = grads
        self.g[:] = [g.data_ptr() for g in grads]


class MultiTensorArgs32(_GradList):
    """Host pointer arrays for ``bwd_adam32_step_multi``, built once for a
    fixed list of tensors and reused by every step."""

    def __init__(self, params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor],
                 m: Sequence[torch.Tensor], v: Sequence[torch.Tensor]):
        if not (len(grads) == len(m) == len(v) == len(params)):
            raise ValueError("all lists must have the same length")
        self.p_dtype = _one_dtype(params, "parameters")
        self.g_dtype = _one_dtype(grads, "gradients")
        self._init_grads(grads, params[0].device if params else None)
        for i, p in enumerate(params):
            _need(p, f"params[{i}]", p.dtype, self._sizes[i], self.device)
            _need(m[i], f"m[{i}]", torch.float32, self._sizes[i], self.device)
            _need(v[i], f"v[{i}]", torch.float32, self._sizes[i], self.device)
        self._keep = (list(params), list(m), list(v))
        self.p, self.m, self.v = _pointers(params), _pointers(m), _pointers(v)

    def step(self, *, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step, grad_scale=None,
             stream=None) -> None:
        """One AdamW step in place.  ``grad_scale``: a float32 CUDA tensor of
        one element that multiplies every gradient, or None for 1; where it is
        not finite the step writes nothing.  ``step``: which one it is, from 1
        on, or a :class:`StepCount`, which the call advances if it writes."""
        if self.T == 0:
            return
        scale = _check_scale(grad_scale, self.device)
        if isinstance(step, StepCount):
            count = _count_on(step, self.device)
            hp = _abi.AdamWHParams(lr, beta1, beta2, eps, weight_decay, 1)
            return _launch("bwd_adam32_step_multi_counted", self.device, stream, self.T, self.p, self.p_dtype, self.g, self.g_dtype,
                           self.m, self.v, self.n, scale, count, ctypes.byref(hp))
        hp = _abi.AdamWHParams(lr, beta1, beta2, eps, weight_decay, int(step))
        _launch("bwd_adam32_step_multi", self.device, stream, self.T, self.p, self.p_dtype, self.g, self.g_dtype, self.m, self.v, self.n,
                scale, ctypes.byref(hp))


def adam32_step_multi(params, grads, m, v, *, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step,
                      grad_scale=None, stream=None) -> None:
    """One AdamW step with fp32 moments over a list of tensors, in place."""
    MultiTensorArgs32(params, grads, m, v).step(lr=lr, beta1=beta1, beta2=beta2, eps=eps, weight_decay=weight_decay,
                                                step=step, grad_scale=grad_scale, stream=stream)


class GradNorm(_GradList):
    """Norm of a fixed list of gradients, of any of the types.  Its workspace and results belong to
    it: calls of one object are made on one stream, or ordered by the caller,
    and each writes the same two tensors again."""

    def __init__(self, grads: Sequence[torch.Tensor], device=None):
        if not grads and device is None:
            raise ValueError("an empty list needs a device")
        self._init_grads(grads, grads[0].device if grads else torch.device(device))
        self._types = (ctypes.c_int32 * self.T)(*[_GDT[d] for d in self._dtypes])
        self.factor = torch.empty(1, dtype=torch.float32, device=self.device)
        self.norm = torch.empty(1, dtype=torch.float32, device=self.device)
        self._work = torch.zeros(_lib.bwd_grad_norm_work_bytes(self.T), dtype=torch.uint8, device=self.device)

    def clip_scale(self, max_norm: float, loss_scale: float = 1.0, stream=None):
        """(factor, norm), the object's float32 CUDA tensors of one element: norm of the
        gradients divided by ``loss_scale``, and the factor that divides by
        ``loss_scale`` and clips to ``max_norm``: min(1, max_norm / (norm +
        1e-6)) / loss_scale, NaN where the norm is not finite."""
        _launch("bwd_grad_norm", self.device, stream, self.T, self.g, self._types, self.n, max_norm, loss_scale,
                self.factor.data_ptr(), self.norm.data_ptr(), self._work.data_ptr())
        return self.factor, self.norm


def clip_scale(grads: Sequence[torch.Tensor], max_norm: float, loss_scale: float = 1.0, stream=None):
    """:meth:`GradNorm.clip_scale` of a list used once."""
    if stream is not None:  # its workspace belongs to the stream that it is used on
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(stream, grads[0].device)
        with torch.cuda.stream(stream):
            return GradNorm(grads).clip_scale(max_norm, loss_scale)
    return GradNorm(grads).clip_scale(max_norm, loss_scale)
