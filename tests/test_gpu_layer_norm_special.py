"""Special rows among many: constant ones, infinities, NaN, offsets and sizes far from one, in both passes."""

import numpy as np
import pytest
import torch

from oracle import layer_norm as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
U = 2.0 ** -24
ROUND = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
TINY = {"fp32": 2.0 ** -149, "bf16": 2.0 ** -134, "fp16": 2.0 ** -25}


@pytest.fixture(scope="module")
def norm():
    from block_wise_dynamic_gb300 import build

    build.build()
    from block_wise_dynamic_gb300 import norm as m

    return m


def np64(t):
    return t.detach().double().cpu().numpy()


def rows_of(rows, width, kind, seed):
    rng = np.random.default_rng(seed)
    return torch.from_numpy(rng.standard_normal((rows, width))).to(DEV, TYPES[kind])


def forward_bound(x, want, m, r, kind):
    """A thread adds up to 32 values one after the other, a CTA up to 16 warps' sums behind 5 more additions: a sum is within 54 U of the sum
    of magnitudes, and what it is divided by within U.  The variance is that of values centred by the mean so found, and twice as
    many roundings; half of its error is rstd's, which takes 2 U more."""
    off_mean = 56 * U * np.abs(x).mean(1)
    off_r = 0.5 * (64 * U + (off_mean * r) ** 2 + 2 * off_mean * r * 4 * U) + 4 * U
    off = (off_mean * r)[:, None] * (1 + 4 * U) + np.abs((x - m[:, None]) * r[:, None]) * (off_r + 4 * U)[:, None]
    off = off + 2 * U * (np.abs(want) + off)
    return off + ROUND[kind] * (np.abs(want) + off) + TINY[kind]


def backward_bound(dy, x, m, r, want, kind):
    xh, h = np.abs((x - m[:, None]) * r[:, None]), np.abs(dy)
    off = r[:, None] * U * (6 * h + 60 * h.mean(1, keepdims=True) + 66 * xh * (h * xh).mean(1, keepdims=True))
    return off + ROUND[kind] * (np.abs(want) + off) + TINY[kind]


# up to 512 columns a warp takes a row, beyond that a CTA; from 8193 on a thread holds more values; 1003 and 9001 are no whole pieces of 16 bytes
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("rows,width", [(4000, 300), (4000, 1000), (4000, 1003), (3000, 1024), (2500, 4096), (1500, 8192), (1500, 9001), (1200, 16384)])
def test_special_rows(norm, rows, width, kind):
    x, dy = rows_of(rows, width, kind, 1), rows_of(rows, width, kind, 2)
    beta = torch.linspace(-1, 1, width, device=DEV)
    plain = norm.forward(x, None, beta)
    last = rows - 1
    big, small = {"fp32": (1e15, 1e-25), "bf16": (1e15, 1e-25), "fp16": (1e3, 1e-4)}[kind]
    x[1] = 3.25
    x[2, 5] = float("inf")
    x[3, width - 1] = float("nan")
    x[4] += {"fp32": 1e4, "bf16": 100.0, "fp16": 100.0}[kind]
    x[5] *= big
    x[6] *= small
    x[7] = 0.0
    x[last - 1] = float("-inf")
    x[last, 0] = float("nan")
    bad = [2, 3, last - 1, last]
    y, mean, rstd = norm.forward(x, None, beta)
    at = beta.to(TYPES[kind])
    assert torch.equal(y[1], at) and torch.equal(y[7], at)
    assert y[bad].isnan().any(1).all() and y[[3, last - 1, last]].isnan().all()
    good = torch.ones(rows, dtype=torch.bool, device=DEV)
    good[bad] = False
    assert y[good].isfinite().all() and mean[good].isfinite().all() and rstd[good].isfinite().all()
    # rows next to special ones are what they are among others
    same = good.clone()
    same[:8] = False
    same[0] = True
    for a, b in zip((y, mean, rstd), plain):
        assert torch.equal(a[same], b[same])
    pick = [0, 1, 4, 5, 6, 7, 8, rows // 2, last - 2]
    xs = np64(x[pick])
    want, m, r = ref.forward(xs, None, np64(beta))
    assert (np.abs(np64(y[pick]) - want) <= forward_bound(xs, want, m, r, kind)).all()

    # backward: a special row's gradient is its own, the columns' sums are theirs
    grads = norm.backward(dy, x, None, mean, rstd)
    dx = grads[0]
    assert dx[[3, last - 1, last]].isnan().all() and dx[good].isfinite().all()
    m, r = np64(mean[pick]), np64(rstd[pick])
    ds = np64(dy[pick])
    want = ref.backward(ds, xs, None, m, r)[0]
    assert (np.abs(np64(dx[pick]) - want) <= backward_bound(ds, xs, m, r, want, kind)).all()
    assert grads[1].isnan().any()
    # the sums of the same rows without the ones that are not finite
    x[bad], dy[bad] = 0.0, 0.0
    y, mean, rstd = norm.forward(x)
    _, dgamma, dbeta = norm.backward(dy, x, None, mean, rstd)
    xs, ds, m, r = np64(x), np64(dy), np64(mean), np64(rstd)
    xh = np.abs((xs - m[:, None]) * r[:, None])
    _, want_g, want_b = ref.backward(ds, xs, None, m, r)
    chain = rows / 152 + 1 + 8 + 160 * 4 / 8 + 8
    for got, want, size in ((dgamma, want_g, (np.abs(ds) * xh).sum(0)), (dbeta, want_b, np.abs(ds).sum(0))):
        assert (np.abs(np64(got) - want) <= U * (chain + 4) * size + U * np.abs(want)).all()


@pytest.mark.parametrize("rows,width", [(4000, 1000), (3000, 1003), (1500, 9001)])
def test_gradients_that_are_not_finite(norm, rows, width):
    """An infinity or a NaN among the incoming gradients stays in its row and its column."""
    x, dy = rows_of(rows, width, "fp32", 3), rows_of(rows, width, "fp32", 4)
    _, mean, rstd = norm.forward(x)
    plain = norm.backward(dy, x, None, mean, rstd)
    dy[7, 3], dy[rows - 1, width - 1] = float("inf"), float("nan")
    dx, dgamma, dbeta = norm.backward(dy, x, None, mean, rstd)
    rest = [i for i in range(rows) if i not in (7, rows - 1)]
    assert torch.equal(dx[rest], plain[0][rest]) and dx[rows - 1].isnan().all() and not dx[7].isfinite().any()
    cols = [i for i in range(width) if i not in (3, width - 1)]
    for a, b in ((dgamma, plain[1]), (dbeta, plain[2])):
        assert torch.equal(a[cols], b[cols]) and not a[3].isfinite() and a[width - 1].isnan()
