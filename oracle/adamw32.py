"""Plain 64-bit statements of AdamW with unquantized moments and of the
gradients' norm and clipping factor, in NumPy."""

from __future__ import annotations

import numpy as np


def step(p, g, m, v, *, lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step, scale=1.0):
    """New (p, m, v), all in binary64."""
    p, g, m, v = (np.asarray(t, np.float64) for t in (p, g, m, v))
    g = g * scale
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    mhat = m / (1 - beta1 ** step)
    vhat = v / (1 - beta2 ** step)
    return p - lr * weight_decay * p - lr * mhat / (np.sqrt(vhat) + eps), m, v


def clip(grads, max_norm, loss_scale=1.0):
    """(factor, norm)."""
    norm = np.sqrt(sum(float(np.sum(np.square(np.asarray(g, np.float64)))) for g in grads)) / loss_scale
    return (min(1.0, max_norm / (norm + 1e-6)) / loss_scale if np.isfinite(norm) else np.nan), norm
