"""First derivatives only: autograd Functions whose backward pass computes
through addresses."""

from __future__ import annotations

from functools import wraps

import torch


class _NoSecondDerivative(torch.autograd.Function):
    """The given gradients, as functions of something: the first argument, a
    tensor that takes a gradient, stands for all that they depend on."""

    @staticmethod
    def forward(ctx, name, anything, *gradients):
        ctx.name = name
        return tuple(g.detach() for g in gradients)  # not views, which could not be changed in place

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError(f"{ctx.name} has no second derivatives")


def first_order(name: str):
    """Decorator of a Function's ``backward``.  With ``create_graph`` its
    results carry a node that raises when something is differentiated through
    them.  (torch's ``once_differentiable`` does so only where an incoming
    gradient takes a gradient itself; these results depend on the saved
    tensors too.)"""

    def decorate(backward):
        @wraps(backward)
        def wrapped(ctx, *gradients):
            with torch.no_grad():
                out = backward(ctx, *gradients)
            if not torch.is_grad_enabled():
                return out
            out = out if isinstance(out, tuple) else (out,)
            some = [g for g in out if g is not None]
            if not some:
                return out
            marked = iter(_NoSecondDerivative.apply(name, torch.empty(0, requires_grad=True), *some))
            return tuple(None if g is None else next(marked) for g in out)

        return wrapped

    return decorate
