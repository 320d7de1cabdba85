"""Pins of the 64-bit statements that the 8-bit products and the 32-bit-state
step are tested against."""

import numpy as np
import pytest
import torch

from oracle import adamw32, fp8


def test_values_are_torchs():
    v = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).to(torch.float64).numpy()
    assert np.array_equal(fp8.e4m3_values(), v, equal_nan=True)


def test_rounding_is_to_the_nearest_value_ties_to_even():
    values = np.unique(fp8.e4m3_values()[~np.isnan(fp8.e4m3_values())])
    mids = (values[1:] + values[:-1]) / 2
    x = np.concatenate([values, mids, np.nextafter(mids, -1e9), np.nextafter(mids, 1e9)])
    got = fp8.round_e4m3(x)
    d = np.abs(x[:, None] - values)
    near = d == d.min(1, keepdims=True)
    assert all(near[i, np.searchsorted(values, got[i])] for i in range(len(x)))
    assert np.array_equal(got[:255 - 2], values[:255 - 2])
    t = torch.from_numpy(x.astype(np.float32))
    same = t.double().numpy() == x  # the points that fp32 holds
    assert np.array_equal(t.to(torch.float8_e4m3fn).double().numpy()[same], got[same])


@pytest.mark.parametrize("a,e", [(448.0, 0), (np.nextafter(np.float32(448), np.float32(1e9)), 1), (0.0, -127), (1.0, -8), (1.75, -8),
                                 (2.0, -7), (2.0 ** -149, -127), (np.float32(3.4028235e38), 120), (np.inf, 128), (np.nan, 128)])
def test_exponent(a, e):
    assert fp8.block_exponents(np.array([[0.0, -a]]), 1, 128)[0, 0] == e


def test_linear_on_representable_values_is_plain():
    rng = np.random.default_rng(0)
    x, w, dy = rng.integers(-8, 9, (5, 300)), rng.integers(-8, 9, (7, 300)), rng.integers(-8, 9, (5, 7))
    y, _ = fp8.linear(x, w, np.arange(7))
    assert np.array_equal(y, x @ w.T + np.arange(7))
    (dx, dw, db), _ = fp8.linear_backward(dy, x, w)
    assert np.array_equal(dx, dy @ w) and np.array_equal(dw, dy.T @ x) and np.array_equal(db, dy.sum(0))


def test_adamw_matches_torch():
    rng = np.random.default_rng(1)
    p = torch.nn.Parameter(torch.from_numpy(rng.standard_normal(50)))
    opt = torch.optim.AdamW([p], lr=1e-2, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)
    q, m, v = p.detach().numpy().copy(), np.zeros(50), np.zeros(50)
    for t in range(1, 6):
        g = rng.standard_normal(50)
        p.grad = torch.from_numpy(2.0 * g)
        opt.step()
        q, m, v = adamw32.step(q, g, m, v, lr=1e-2, beta2=0.99, weight_decay=0.1, step=t, scale=2.0)
    np.testing.assert_allclose(q, p.detach().numpy(), rtol=1e-12)


def test_clip_matches_torch():
    rng = np.random.default_rng(2)
    gs = [rng.standard_normal(n) for n in (3, 40)]
    ps = [torch.nn.Parameter(torch.zeros(len(g), dtype=torch.float64)) for g in gs]
    for p, g in zip(ps, gs):
        p.grad = torch.from_numpy(g.copy())
    norm = torch.nn.utils.clip_grad_norm_(ps, 0.5)
    factor, mine = adamw32.clip(gs, 0.5)
    np.testing.assert_allclose(mine, norm.item(), rtol=1e-12)
    np.testing.assert_allclose(ps[1].grad.numpy(), gs[1] * factor, rtol=1e-12)
    assert adamw32.clip([np.array([3.0, 4.0])], 1e9, 2.0) == (0.5, 2.5)
    assert np.isnan(adamw32.clip([np.array([np.inf])], 1.0)[0])
