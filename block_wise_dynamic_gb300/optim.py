"""Drop-in replacement for ``torch.optim.Adam`` with 8-bit block-wise states.

The page on "8-BIT OPTIMIZERS VIA BLOCK-WISE QUANTIZATION" says switching to
the 8-bit optimizer takes two lines of code (introduction and 总结); this
class is that switch:

    from block_wise_dynamic_gb300 import Adam8bit
    opt = Adam8bit(model.parameters(), lr=1e-3, betas=(0.9, 0.999), eps=1e-8)

``AdamW8bit`` is the same with decoupled weight decay.

Parameters are fp32 (master weights), bf16 or fp16 CUDA tensors (widened for
the update, stored back rounded to nearest even); gradients fp32, bf16 or
fp16.  Per parameter the state holds ``step`` and the codes and absmax of
both moments; ``state_dict()`` / ``load_state_dict()`` round-trip them
exactly.  Each ``step()`` issues one multi-tensor launch per (device,
gradient dtype, step count) group.  A parameter group with ``state_bits=32``
(an embedding, norms, biases) keeps its moments in fp32 (``exp_avg``,
``exp_avg_sq``) and takes the 32-bit step.  ``clip_scale`` computes the norm
of all gradients and the clipping factor on the device, and ``step`` takes
that factor:

    factor, norm = opt.clip_scale(1.0)
    opt.step(grad_scale=factor)

The launch tables are built once per
parameter group and reused: when gradients are fresh tensors each step (the
default ``zero_grad(set_to_none=True)``), a step only re-reads the gradient
pointers.
"""

from __future__ import annotations

from collections import defaultdict

import torch

from . import GradNorm, MultiTensorArgs, MultiTensorArgs32, StepCount, num_blocks, state_init


class _Counts:
    """Step counts of states as numbers; one that lies on the device, which
    many states share, is read once."""

    def __init__(self):
        self._read = {}

    def __call__(self, state) -> int:
        step = state["step"]
        if not torch.is_tensor(step):
            return step
        if id(step) not in self._read:
            self._read[id(step)] = step, int(step)
        return self._read[id(step)][1]


class Adam8bit(torch.optim.Optimizer):
    """8-bit Adam (``weight_decay`` must be 0: torch.optim.Adam's coupled L2
    decay is not part of this step; use :class:`AdamW8bit` for decay)."""

    _decoupled = False

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0, state_bits=8):
        if lr < 0.0:
            raise ValueError(f"invalid learning rate {lr}")
        if not (0.0 <= betas[0] < 1.0 and 0.0 <= betas[1] < 1.0):
            raise ValueError(f"invalid betas {betas}")
        if eps < 0.0:
            raise ValueError(f"invalid eps {eps}")
        if weight_decay < 0.0 or (weight_decay != 0.0 and not self._decoupled):
            raise ValueError("Adam8bit takes no weight decay; AdamW8bit applies it decoupled")
        super().__init__(params, dict(lr=lr, betas=betas, eps=eps, weight_decay=weight_decay, state_bits=state_bits))
        self._args_cache = {}
        self._norm = None

    def __setstate__(self, state):
        # a copied or unpickled optimizer has none of the launch tables; their addresses were the original's
        super().__setstate__(state)
        self._args_cache = {}
        self._norm = None

    def add_param_group(self, param_group):
        if isinstance(param_group, dict) and param_group.get("state_bits", self.defaults["state_bits"]) not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        super().add_param_group(param_group)

    def _state_for(self, p: torch.Tensor, bits: int):
        st = self.state[p]
        if len(st) == 0 and bits == 32:
            st["step"] = 0
            st["exp_avg"] = torch.zeros(p.numel(), dtype=torch.float32, device=p.device)
            st["exp_avg_sq"] = torch.zeros(p.numel(), dtype=torch.float32, device=p.device)
        elif len(st) == 0:
            mc, ma, vc, va = state_init(p.numel(), p.device)
            st["step"] = 0
            st["m_codes"], st["m_absmax"], st["v_codes"], st["v_absmax"] = mc, ma, vc, va
        return st

    def _plan(self, params, grads, bits):
        """Launch plan of one parameter group: its parameters with a gradient,
        bucketed by (device, parameter dtype, gradient dtype, step count), each
        bucket with its argument table (parameter and state pointers fixed)."""
        buckets = defaultdict(list)
        count = _Counts()
        for i, (p, g) in enumerate(zip(params, grads)):
            if g is None:
                continue
            if p.dtype not in (torch.float32, torch.bfloat16, torch.float16) or not p.is_cuda:
                raise TypeError("Adam8bit needs fp32, bf16 or fp16 CUDA parameters")
            if g.is_sparse:
                raise TypeError("sparse gradients are not supported")
            st = self._state_for(p, bits)
            if ("exp_avg" in st) != (bits == 32):
                raise ValueError(f"the state of a parameter is not the one of state_bits={bits}")
            if bits == 8 and st["m_absmax"].numel() != num_blocks(p.numel()):
                raise ValueError("state does not match the parameter size")
            buckets[(p.device, p.dtype, g.dtype, count(st))].append(i)
        plan = []
        for (_, _, _, t), idx in buckets.items():
            sts = [self.state[params[i]] for i in idx]
            gs = [grads[i] if grads[i].is_contiguous() else grads[i].contiguous() for i in idx]
            lists = [params[i].view(-1) for i in idx], [g.view(-1) for g in gs]
            if bits == 32:
                args = MultiTensorArgs32(*lists, [s["exp_avg"].view(-1) for s in sts], [s["exp_avg_sq"].view(-1) for s in sts])
            else:
                args = MultiTensorArgs(*lists, [s["m_codes"] for s in sts], [s["m_absmax"] for s in sts],
                                       [s["v_codes"] for s in sts], [s["v_absmax"] for s in sts])
            plan.append([idx, sts, args, t])
        for _, sts, _, t in plan:
            for s in sts:
                s["step"] = t
        return {"params": list(params), "has_grad": [g is not None for g in grads], "buckets": plan}

    @torch.no_grad()
    def clip_scale(self, max_norm: float, loss_scale: float = 1.0):
        """(factor, norm) of all gradients as new one-element CUDA tensors (see
        :meth:`GradNorm.clip_scale`); pass the factor to :meth:`step`.  Where
        the norm is not finite the factor is NaN and that step writes no
        parameter and no moment and is not counted."""
        grads = [p.grad for group in self.param_groups for p in group["params"] if p.grad is not None]
        if not grads:
            raise ValueError("no parameter has a gradient")
        if any(g.is_sparse for g in grads):
            raise TypeError("sparse gradients are not supported")
        grads = [g if g.is_contiguous() else g.contiguous() for g in grads]
        try:
            if self._norm is None:
                raise ValueError
            self._norm.set_grads(grads)
        except (TypeError, ValueError):  # the first call, or other gradients than before
            self._norm = GradNorm(grads)
        # results of this call's own: the object would write an earlier call's again
        self._norm.factor, self._norm.norm = torch.empty((2, 1), dtype=torch.float32, device=self._norm.device).unbind()
        return self._norm.clip_scale(max_norm, loss_scale)

    @torch.no_grad()
    def step(self, closure=None, grad_scale=None):
        """One step.  ``grad_scale``: a one-element float32 CUDA tensor that
        multiplies every gradient, or None.  Where it is not finite the step
        writes nothing and is not counted; from the first call with one on,
        the states' ``step`` is therefore an int64 CUDA tensor (a number again
        in ``state_dict()``), and a step captured in a graph after that is
        replayed as the next one."""
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        for gi, group in enumerate(self.param_groups):
            params = group["params"]
            grads = [p.grad for p in params]
            plan = self._args_cache.get(gi)
            fresh = (plan is None or len(plan["params"]) != len(params)
                     or not all(a is b for a, b in zip(plan["params"], params))
                     or plan["has_grad"] != [g is not None for g in grads])
            if fresh:
                plan = self._args_cache[gi] = self._plan(params, grads, group.get("state_bits", 8))
            b1, b2 = group["betas"]
            for bucket in plan["buckets"]:
                idx, sts, args, t = bucket
                if not fresh:
                    try:
                        args.set_grads([grads[i] for i in idx])
                    except (TypeError, ValueError):
                        # a gradient changed dtype or shape: rebuild this group's plan next step
                        self._args_cache.pop(gi, None)
                        raise
                counted = isinstance(t, StepCount)
                if grad_scale is not None and not counted:
                    t, counted = StepCount(args.device, t), True
                args.step(lr=group["lr"], beta1=b1, beta2=b2, eps=group["eps"], weight_decay=group["weight_decay"],
                          step=t if counted else t + 1, grad_scale=grad_scale)
                # the step count advances only once its launch went through
                if not counted:
                    t += 1
                if t is not bucket[3]:
                    bucket[3] = t
                    for s in sts:
                        s["step"] = t.taken if counted else t
        return loss

    def _reset_plans(self):
        """Forget the cached launch plans (after the state was replaced)."""
        self._args_cache = {}

    def state_dict(self):
        sd = super().state_dict()
        count = _Counts()
        sd["state"] = {k: {**st, "step": count(st)} if "step" in st else st for k, st in sd["state"].items()}
        return sd

    def load_state_dict(self, state_dict):
        self._reset_plans()
        super().load_state_dict(state_dict)
        # torch casts every floating parameter's state tensors to the
        # parameter dtype: codes are integers 0..255, so casting back is
        # exact, and fp32 tensors are taken again from the saved ones
        saved = state_dict["state"]
        order = [p for g in self.param_groups for p in g["params"]]
        ids = [i for g in state_dict["param_groups"] for i in g["params"]]
        for i, p in zip(ids, order):
            if i not in saved or p not in self.state:
                continue
            st = self.state[p]
            for k in ("m_codes", "v_codes"):
                if k in st and st[k].dtype != torch.uint8:
                    st[k] = st[k].to(torch.uint8)
            for k in ("m_absmax", "v_absmax", "exp_avg", "exp_avg_sq"):
                if k in st and st[k].dtype != torch.float32:
                    st[k] = saved[i][k].to(device=p.device, dtype=torch.float32, copy=True)


class AdamW8bit(Adam8bit):
    """8-bit AdamW: decoupled weight decay, p <- p * (1 - lr * weight_decay)
    before the Adam update (torch.optim.AdamW's rule)."""

    _decoupled = True

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=1e-2, state_bits=8):
        super().__init__(params, lr=lr, betas=betas, eps=eps, weight_decay=weight_decay, state_bits=state_bits)
