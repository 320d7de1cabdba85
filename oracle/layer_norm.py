"""Layer normalisation over rows in binary64, forward and backward."""

from __future__ import annotations

import numpy as np


def forward(x, gamma=None, beta=None, eps=1e-5):
    """(y, mean, rstd) of the rows of x."""
    x = np.asarray(x, np.float64)
    mean = x.mean(1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    y = (x - mean[:, None]) * rstd[:, None]
    if gamma is not None:
        y = y * gamma
    return (y if beta is None else y + beta), mean, rstd


def backward(dy, x, gamma, mean, rstd):
    """(dx, dgamma, dbeta) for the given statistics."""
    dy = np.asarray(dy, np.float64)
    xh = (np.asarray(x, np.float64) - mean[:, None]) * rstd[:, None]
    h = dy if gamma is None else dy * gamma
    dx = rstd[:, None] * (h - h.mean(1, keepdims=True) - xh * (h * xh).mean(1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0)
