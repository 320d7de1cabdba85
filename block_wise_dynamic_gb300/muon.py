"""Orthogonalised updates for matrices, next to Adam for everything else.

A matrix's update is its momentum with all singular values brought towards 1
by Newton-Schulz steps:

  X = G / (|G| + 1e-7);  5 times:  A = X X^T;  X = a X + (b A + c A A) X

with (a, b, c) = (3.4445, -4.7750, 2.0315).

  orthogonalize(g)                  X of one matrix, or of each of a batch
  MuonArgs(params, grads, momenta)  pointer tables of a fixed list; .step()
  Muon                              torch.optim.Optimizer for matrices

    opt = Muon([p for p in blocks.parameters() if p.ndim == 2], lr=0.02)
    rest = AdamW8bit(others, lr=1e-3)

Each call checks and marshals CUDA tensors and makes one call into
``libbwd.so`` (``bwd_orthogonalize``, ``bwd_muon_step`` in ``include/bwd.h``);
the products run on the tensor cores on pairs of fp16 values.
"""

from __future__ import annotations

import ctypes
from typing import Sequence

import torch

from . import _abi
from . import _GDT, _launch, _lib, _need, _stream_handle
from .adam32 import _check_scale, _GradList, _one_dtype, _pointers
from .fp8 import _on
from .optim import Adam8bit

__all__ = ["orthogonalize", "MuonArgs", "Muon"]


def _sides(shapes):
    kind = ctypes.c_int64 * len(shapes)
    return kind(*[r for r, _ in shapes]), kind(*[c for _, c in shapes])


def _work_bytes(count, rows, cols, most=0):
    size = _lib.bwd_muon_work_bytes(count, rows, cols, most)
    if size < 0:
        raise ValueError("a matrix has at most 65536 rows and columns")
    return size


def orthogonalize(g: torch.Tensor, steps: int = 5, stream=None) -> torch.Tensor:
    """``g`` (..., rows, columns; float32, bfloat16 or float16), each matrix
    orthogonalised, in its type.  A matrix of zeros stays one; one with a NaN
    or an infinity comes out NaN.  bfloat16 matrices with two to sixteen times
    as many columns as rows, or the other way round, take a faster form that is
    up to 1e-4 off beside their rounding's 1.7e-3; ``g.float()`` takes the more
    exact one."""
    if not isinstance(g, torch.Tensor):
        raise TypeError("g must be a torch.Tensor")
    if not g.is_cuda:
        raise ValueError("g must be a CUDA tensor")
    if g.dtype not in _GDT:
        raise TypeError("g must be float32, bfloat16 or float16")
    if g.dim() < 2:
        raise ValueError("g must have rows and columns")
    if stream is not None:
        with _on(stream, g.device):
            return orthogonalize(g, steps)
    g = g.contiguous()
    out = torch.empty_like(g)
    r, c = g.shape[-2:]
    count = g.numel() // (r * c) if r * c else 0
    if count == 0:
        return out
    rows, cols = _sides([(r, c)] * count)
    work = torch.empty(_work_bytes(count, rows, cols), dtype=torch.uint8, device=g.device)
    size = r * c * g.element_size()
    table = ctypes.c_void_p * count
    _launch("bwd_orthogonalize", g.device, None, count, table(*[g.data_ptr() + i * size for i in range(count)]), _GDT[g.dtype], rows, cols,
            int(steps), table(*[out.data_ptr() + i * size for i in range(count)]), work.data_ptr())
    return out


class MuonArgs(_GradList):
    """Host pointer arrays for ``bwd_muon_step``, built once for a fixed list
    of matrices and reused by every step.  Its workspace belongs to it and to
    the stream of its first step (or is ``work``, that of another list made on
    the stream that is current now, if it is as large); a step on another
    stream, or in a graph that is captured, takes one of its own.  Matrices
    are worked on together, up to 64 at a time and as far as ``work_bytes`` of
    workspace hold them, 4 GB by default (a matrix of m x n takes 8 m (m + n)
    to 8 m (2 m + n) bytes, m its shorter side): less memory in more, smaller
    launches."""

    def __init__(self, params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor], momenta: Sequence[torch.Tensor], work=None, work_bytes=None):
        if work_bytes is not None and not 0 < work_bytes < 1 << 63:
            raise ValueError("work_bytes must be a positive number of bytes")
        if not (len(grads) == len(momenta) == len(params)):
            raise ValueError("all lists must have the same length")
        self.p_dtype = _one_dtype(params, "parameters")
        self.g_dtype = _one_dtype(grads, "gradients")
        self._init_grads(grads, params[0].device if params else None)
        for i, p in enumerate(params):
            _need(p, f"params[{i}]", p.dtype, self._sizes[i], self.device)
            if p.dim() != 2:
                raise ValueError(f"params[{i}] must be a matrix")
            if grads[i].shape != p.shape:
                raise ValueError(f"grads[{i}] must have its parameter's shape")
            _need(momenta[i], f"momenta[{i}]", torch.float32, self._sizes[i], self.device)
        self._keep = (list(params), list(momenta))
        self.p, self.m = _pointers(params), _pointers(momenta)
        self._shapes = [p.shape for p in params]
        self.rows, self.cols = _sides(self._shapes)
        self._held = self._stream = None
        if self.T:
            self._most = int(work_bytes or 0)
            self._size = _work_bytes(self.T, self.rows, self.cols, self._most)
            if work is not None and work.device == self.device and work.is_contiguous() and work.nbytes >= self._size:
                self._held, self._stream = work, _stream_handle(self.device, None)

    @property
    def work(self):
        """The list's workspace; the first access makes it, on the stream that is current."""
        if self._held is None and self.T:
            self._held, self._stream = self._new_work(), _stream_handle(self.device, None)
        return self._held

    def _new_work(self):
        return torch.empty(self._size, dtype=torch.uint8, device=self.device)

    def set_grads(self, grads: Sequence[torch.Tensor]) -> None:
        if [g.shape for g in grads] != self._shapes:
            raise ValueError("gradient shapes differ from the parameters'")
        super().set_grads(grads)

    def _workspace(self, stream):
        """The list's workspace, or one for a single call: the memory of the
        list's follows the order of the stream that it was made on alone, and a
        graph may outlive it."""
        if stream is not None:
            with _on(stream, self.device):
                return self._workspace(None)
        if torch.cuda.is_current_stream_capturing() or self._held is not None and self._stream != _stream_handle(self.device, None):
            return self._new_work()
        return self.work

    def step(self, *, lr=0.02, momentum=0.95, nesterov=True, weight_decay=0.0, rms=0.2, steps=5, grad_scale=None, stream=None) -> None:
        """One step in place:

          m = momentum m + s g;  u = s g + momentum m (nesterov), or m
          p = p (1 - lr weight_decay) - lr rms sqrt(max(p.shape)) orthogonalize(u)

        ``rms``: root mean square that a full-rank update has before lr.
        ``grad_scale``: s, a float32 CUDA tensor of one element, or None for
        1; where it is not finite the step writes nothing."""
        if self.T == 0:
            return
        hp = _abi.MuonHParams(lr, momentum, weight_decay, rms, int(bool(nesterov)), int(steps), self._most)
        scale, work = _check_scale(grad_scale, self.device), self._workspace(stream)
        _launch("bwd_muon_step", self.device, stream, self.T, self.p, self.p_dtype, self.g, self.g_dtype, self.m, self.rows, self.cols,
                scale, ctypes.byref(hp), work.data_ptr())


class Muon(torch.optim.Optimizer):
    """Momentum and orthogonalised updates for parameters of two or more
    dimensions (those after the first are taken together).  Parameters and
    gradients are float32, bfloat16 or float16 CUDA tensors, momentum float32;
    the update is formed to some 17 to 20 bits, to 13 of bfloat16 parameters
    with two to sixteen times as many columns as rows, or the other way round.
    ``clip_scale`` and ``step(grad_scale=factor)`` are as :class:`Adam8bit`'s.
    The steps of all groups share a workspace for each device and stream; one
    that is captured in a graph takes one of its own.  It lives as long as the
    optimizer; ``work_bytes`` limits it, to 4 GB by default (see
    :class:`MuonArgs`): 48 matrices of 1024 x 4096 take 2.4 GB, or 1.2 with 2 GB
    for a limit, and 4% more time."""

    def __init__(self, params, lr=0.02, momentum=0.95, nesterov=True, weight_decay=0.0, rms=0.2, steps=5, work_bytes=None):
        if not 0.0 <= lr < float("inf"):
            raise ValueError(f"invalid learning rate {lr}")
        if not 0.0 <= momentum < 1.0:
            raise ValueError(f"invalid momentum {momentum}")
        if not 0.0 <= weight_decay < float("inf") or not 0.0 <= rms < float("inf"):
            raise ValueError("weight_decay and rms must be finite and >= 0")
        if not 1 <= steps <= 100:
            raise ValueError("steps must be 1 to 100")
        if work_bytes is not None and not 0 < work_bytes < 1 << 63:
            raise ValueError("work_bytes must be a positive number of bytes")
        super().__init__(params, dict(lr=lr, momentum=momentum, nesterov=nesterov, weight_decay=weight_decay, rms=rms, steps=steps,
                                      work_bytes=work_bytes))
        self._reset_plans()

    def __setstate__(self, state):
        # a copied or unpickled optimizer has none of the pointer tables; their addresses were the original's
        super().__setstate__(state)
        self._reset_plans()

    def _reset_plans(self):
        self._args_cache, self._work, self._norm = {}, {}, None

    def add_param_group(self, param_group):
        super().add_param_group(param_group)
        for p in self.param_groups[-1]["params"]:
            if p.dim() < 2:
                self.param_groups.pop()
                raise ValueError("Muon takes matrices; vectors go to another optimizer")

    clip_scale = Adam8bit.clip_scale

    def _plan(self, params, grads, work_bytes):
        buckets = {}
        for i, (p, g) in enumerate(zip(params, grads)):
            if g is None or p.numel() == 0:
                continue
            if p.dtype not in _GDT or not p.is_cuda:
                raise TypeError("Muon needs fp32, bf16 or fp16 CUDA parameters")
            if g.is_sparse:
                raise TypeError("sparse gradients are not supported")
            if not p.is_contiguous():
                raise ValueError("Muon needs contiguous parameters")
            if "momentum_buffer" not in self.state[p]:
                if torch.cuda.is_current_stream_capturing():
                    raise RuntimeError("a parameter's first step makes its momentum and cannot be captured: each replay would make it again")
                self.state[p]["momentum_buffer"] = torch.zeros(p.shape, dtype=torch.float32, device=p.device)
            buckets.setdefault((p.device, p.dtype, g.dtype), []).append(i)
        plan = []
        for (device, _, _), idx in buckets.items():
            ps = [params[i].view(params[i].shape[0], -1) for i in idx]
            place = device, _stream_handle(device, None)
            args = MuonArgs(ps, self._matrices(grads, idx), [self.state[params[i]]["momentum_buffer"] for i in idx], self._work.get(place),
                            work_bytes)
            if not torch.cuda.is_current_stream_capturing():
                self._work[place] = args.work
            plan.append((idx, args))
        return {"params": list(params), "has_grad": [g is not None for g in grads], "at": [p.data_ptr() for p in params],
                "work_bytes": work_bytes, "buckets": plan}

    @staticmethod
    def _matrices(grads, idx):
        return [grads[i].contiguous().view(grads[i].shape[0], -1) for i in idx]

    @torch.no_grad()
    def step(self, closure=None, grad_scale=None):
        """One step.  ``grad_scale``: a one-element float32 CUDA tensor that
        multiplies every gradient, or None; where it is not finite the step
        writes nothing."""
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        for gi, group in enumerate(self.param_groups):
            params = group["params"]
            grads = [p.grad for p in params]
            plan, work_bytes = self._args_cache.get(gi), group.get("work_bytes")  # (none in an older state)
            fresh = (plan is None or plan["work_bytes"] != work_bytes or len(plan["params"]) != len(params) or not all(a is b for a, b in zip(plan["params"], params))
                     or plan["has_grad"] != [g is not None for g in grads] or plan["at"] != [p.data_ptr() for p in params])
            if fresh:
                plan = self._args_cache[gi] = self._plan(params, grads, work_bytes)
            for idx, args in plan["buckets"]:
                if not fresh:
                    try:
                        args.set_grads(self._matrices(grads, idx))
                    except (TypeError, ValueError):
                        # a gradient changed its type: the next step makes a new plan
                        self._args_cache.pop(gi, None)
                        raise
                args.step(lr=group["lr"], momentum=group["momentum"], nesterov=group["nesterov"], weight_decay=group["weight_decay"],
                          rms=group["rms"], steps=group["steps"], grad_scale=grad_scale)
        return loss

    def load_state_dict(self, state_dict):
        self._reset_plans()
        super().load_state_dict(state_dict)
        # torch casts a floating parameter's state to its type: the momentum is taken again from the saved one
        order = [p for g in self.param_groups for p in g["params"]]
        ids = [i for g in state_dict["param_groups"] for i in g["params"]]
        for i, p in zip(ids, order):
            if i in state_dict["state"] and "momentum_buffer" in state_dict["state"][i]:
                saved = state_dict["state"][i]["momentum_buffer"]
                self.state[p]["momentum_buffer"] = saved.to(device=p.device, dtype=torch.float32, copy=True)
