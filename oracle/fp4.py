"""Plain 64-bit statement of microscaled e2m1 quantization and of the product
of two quantized matrices, in NumPy.

A block of 1 x 32 elements has the scale 2^e with the smallest e >= -127 for
which no magnitude exceeds 6 * 2^e; an element's code is the e2m1 value
nearest to x 2^-e, ties to the even code.  A block with an infinity or a NaN
is NaN throughout.
"""

from __future__ import annotations

from fractions import Fraction

import numpy as np

BLOCK = 32
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def exponent(a: float) -> int:
    """The smallest e >= -127 with a <= 6 * 2^e."""
    e = -127
    if a > 0:
        e = max(e, int(np.frexp(a)[1]) - 4)  # a >= 2^(p - 1) > 6 * 2^(p - 4) ... start at or below
        while Fraction(a) > 6 * Fraction(2) ** e:
            e += 1
    return e


def round_code(x) -> np.ndarray:
    """Index into GRID nearest to |x| <= 6, ties to the even index."""
    a = np.abs(np.asarray(x, np.float64))[..., None]
    distance = np.abs(a - GRID)
    least = distance.min(-1, keepdims=True)
    near = distance == least
    even = near & (np.arange(8) % 2 == 0)
    pick = np.where(even.any(-1, keepdims=True), even, near)
    return pick.argmax(-1)


def quantize(x):
    """(values, e): what the codes stand for, and each block's exponent (128
    for a block that is not finite)."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    blocks = -(-cols // BLOCK)
    e = np.zeros((rows, blocks), np.int64)
    out = np.empty_like(x)
    for r in range(rows):
        for b in range(blocks):
            at = slice(BLOCK * b, BLOCK * (b + 1))
            part = x[r, at]
            if not np.isfinite(part).all():
                e[r, b], out[r, at] = 128, np.nan
                continue
            e[r, b] = exponent(np.abs(part).max())
            s = 2.0 ** float(e[r, b])
            out[r, at] = np.copysign(GRID[round_code(part / s)] * s, part)
    return out, e


def linear(x, w, bias=None):
    """(y, magnitude): Q(x) Q(w)^T + bias, and the sum of its terms' magnitudes."""
    qx, qw = quantize(x)[0], quantize(w)[0]
    y, size = qx @ qw.T, np.abs(qx) @ np.abs(qw).T
    return (y, size) if bias is None else (y + bias, size + np.abs(bias))
