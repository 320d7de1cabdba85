"""Newton-Schulz orthogonalisation and the optimizer step on it, in binary64."""

from __future__ import annotations

import numpy as np

A, B, C, EPS = 3.4445, -4.7750, 2.0315, 1e-7


def iterates(g, steps=5):
    """X before each step and after the last, in the wide orientation."""
    x = np.asarray(g, np.float64)
    x = x.T if x.shape[0] > x.shape[1] else x
    out = [x / (np.sqrt((x * x).sum()) + EPS)]
    for _ in range(steps):
        x = out[-1]
        gram = x @ x.T
        out.append(A * x + (B * gram + C * gram @ gram) @ x)
    return out


def orthogonalize(g, steps=5):
    x = iterates(g, steps)[-1]
    return x.T if g.shape[0] > g.shape[1] else x


def step(p, g, m, *, lr, momentum, nesterov=True, weight_decay=0.0, rms=0.2, steps=5, scale=1.0):
    """New parameter and momentum, and the update that was orthogonalised."""
    g = scale * np.asarray(g, np.float64)
    m = momentum * np.asarray(m, np.float64) + g
    u = g + momentum * m if nesterov else m
    p = np.asarray(p, np.float64) * (1 - lr * weight_decay) - lr * rms * np.sqrt(max(u.shape)) * orthogonalize(u, steps)
    return p, m, u
