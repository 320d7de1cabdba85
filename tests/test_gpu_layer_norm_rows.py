"""Layer norm of many rows: what a row gives does not depend on the kernel that takes it."""

import numpy as np
import pytest
import torch

from oracle import layer_norm as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
U = 2.0 ** -24


@pytest.fixture(scope="module")
def norm():
    from block_wise_dynamic_gb300 import build

    build.build()
    from block_wise_dynamic_gb300 import norm as m

    return m


def np64(t):
    return t.detach().double().cpu().numpy()


WIDTHS = [100, 700, 1000, 1003, 1024, 4096, 6000, 8200, 12001, 16384]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("width", WIDTHS)
def test_constant_rows(norm, width, kind):
    """A sum of equal whole numbers is exact below 2^24, its mean then the number, and y beta: with one row, and with many."""
    value = {"fp32": 1000.0, "bf16": 1000.0, "fp16": 1001.0}[kind]
    beta = torch.linspace(-1, 1, width, device=DEV)
    for rows in (1, 9, 4000):
        x = torch.full((rows, width), value, dtype=TYPES[kind], device=DEV)
        x[rows // 2:rows // 2 + 1] = -3.25
        y, mean, rstd = norm.forward(x, None, beta, 1e-5)
        assert torch.equal(y, beta.to(TYPES[kind]).expand(rows, width))
        assert ((mean == value) | (mean == -3.25)).all()
        # less than a unit off
        assert (np.abs(np64(rstd) * float(np.float32(1e-5)) ** 0.5 - 1) < 2 * U).all() and (rstd == rstd[0]).all()


@pytest.mark.parametrize("width", WIDTHS)
def test_exact_statistics(norm, width):
    """Rows of whole numbers whose sums are exact in any order: the same statistics and results with few rows and with many."""
    rng = np.random.default_rng(width)
    half = rng.integers(-8, 9, (40, width // 2))
    x = np.concatenate([half, -half, np.zeros((40, width % 2), np.int64)], 1)  # sums to nothing: the centred values are the values
    x = torch.from_numpy(x).to(DEV, torch.float32)
    var = (np64(x) ** 2).sum(1).astype(np.float32) / np.float32(width)
    want = 1 / np.sqrt((var + np.float32(1e-5)).astype(np.float64))
    many = x.repeat(100, 1)
    few, all_ = (norm.forward(t) for t in (x[:4].contiguous(), many))
    assert not few[1].any() and not all_[1].any()
    assert (np.abs(np64(all_[2]) / np.tile(want, 100) - 1) < 2 * U).all()
    assert torch.equal(few[2], all_[2][:4]) and torch.equal(few[0], all_[0][:4])
    # the backward pass: whole numbers too
    dy = torch.from_numpy(rng.integers(-4, 5, (40, width))).to(DEV, torch.float32)
    one = torch.ones(4, device=DEV)
    zero = torch.zeros(4, device=DEV)
    dx = norm.backward(dy[:4].contiguous(), x[:4].contiguous(), None, zero, one, need_gamma=False, need_beta=False)[0]
    dxs = norm.backward(dy.repeat(100, 1), many, None, torch.zeros(4000, device=DEV), torch.ones(4000, device=DEV), need_gamma=False, need_beta=False)[0]
    assert torch.equal(dx, dxs[:4]) and torch.equal(dxs[:40], dxs[3960:])
