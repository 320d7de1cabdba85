"""Plain 64-bit statement of block-scaled e4m3 quantization and of the linear
layer on quantized operands, in NumPy.

A block's scale is 2^e with the smallest e >= -127 for which no magnitude of
the block exceeds 448 * 2^e; an element's code is the e4m3 value nearest to
x 2^-e, ties to even.  A block with an infinity or a NaN is NaN throughout.
"""

from __future__ import annotations

import numpy as np

BLOCK = 128
MAX = 448.0


def e4m3_values() -> np.ndarray:
    """The 256 values in code order: sign, four exponent bits (bias 7), three
    fraction bits, no infinities, the two codes of all ones NaN."""
    out = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v = np.nan if (c & 127) == 127 else (f / 8) * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        out[c] = -v if c & 128 else v
    return out


def round_e4m3(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value to |x| <= 448, ties to even."""
    x = np.asarray(x, np.float64)
    _, p = np.frexp(x)                              # |x| = f 2^p, f in [0.5, 1)
    grain = np.exp2(np.maximum(p - 1, -6).astype(np.float64) - 3)
    return np.round(x / grain) * grain              # np.round is half to even


def block_exponents(x: np.ndarray, rows: int, cols: int) -> np.ndarray:
    """e of each rows x cols block (partial ones at the edges), 128 for a
    block that is not finite."""
    x = np.asarray(x, np.float64)
    r, c = x.shape
    out = np.zeros((-(-r // rows), -(-c // cols)), np.int64)
    for i in range(out.shape[0]):
        for j in range(out.shape[1]):
            b = np.abs(x[i * rows:(i + 1) * rows, j * cols:(j + 1) * cols])
            if not np.all(np.isfinite(b)):
                out[i, j] = 128
                continue
            a = b.max()
            e = -127
            if a > 0:
                f, p = np.frexp(a / MAX)            # exact: the quotient is compared with powers of two only
                e = max(-127, int(p) - 1 if f == 0.5 else int(p))
                while a > MAX * 2.0 ** e:
                    e += 1
                while e > -127 and a <= MAX * 2.0 ** (e - 1):
                    e -= 1
            out[i, j] = e
    return out


def quantize(x: np.ndarray, rows: int, cols: int):
    """(values, exponents) of a matrix quantized in rows x cols blocks."""
    x = np.asarray(x, np.float64)
    e = block_exponents(x, rows, cols)
    full = np.repeat(np.repeat(e, rows, 0), cols, 1)[:x.shape[0], :x.shape[1]]
    bad = full == 128
    with np.errstate(invalid="ignore", over="ignore"):
        q = np.where(bad, 0.0, x) * np.exp2(-np.where(bad, 0, full).astype(np.float64))
        v = round_e4m3(q) * np.exp2(np.where(bad, 0, full).astype(np.float64))
    return np.where(bad, np.nan, v), e


def linear(x, w, bias=None):
    """(y, sum of the products' magnitudes) for y = Q(x) Q(w)^T + bias."""
    xq, _ = quantize(x, 1, BLOCK)
    wq, _ = quantize(w, BLOCK, BLOCK)
    y = xq @ wq.T
    return (y if bias is None else y + np.asarray(bias, np.float64)), np.abs(xq) @ np.abs(wq).T


def linear_backward(dy, x, w):
    """(dx, dw, dbias) and the sums of magnitudes of the first two."""
    wq, _ = quantize(w, BLOCK, BLOCK)
    dr, _ = quantize(dy, 1, BLOCK)
    dc, _ = quantize(dy, BLOCK, 1)
    xc, _ = quantize(x, BLOCK, 1)
    return (dr @ wq, dc.T @ xc, np.asarray(dy, np.float64).sum(0)), (np.abs(dr) @ np.abs(wq), np.abs(dc).T @ np.abs(xc))
