"""The 64-bit Newton-Schulz statement against the singular value decomposition."""

import numpy as np
import pytest

from oracle import muon as ref


@pytest.mark.parametrize("shape", [(1, 1), (1, 7), (5, 5), (12, 30), (30, 12)])
@pytest.mark.parametrize("steps", [1, 5])
def test_the_steps_act_on_singular_values(shape, steps):
    g = np.random.default_rng(0).standard_normal(shape)
    u, s, vt = np.linalg.svd(g, full_matrices=False)
    s = s / (np.linalg.norm(g) + ref.EPS)
    for _ in range(steps):
        s = ref.A * s + ref.B * s ** 3 + ref.C * s ** 5
    np.testing.assert_allclose(ref.orthogonalize(g, steps), (u * s) @ vt, atol=1e-12)


def test_full_rank_comes_close_to_orthogonal():
    # singular values of a wide Gaussian matrix are all far above 1e-3 of its norm
    x = ref.orthogonalize(np.random.default_rng(1).standard_normal((20, 80)))
    s = np.linalg.svd(x, compute_uv=False)
    assert 0.65 < s.min() and s.max() < 1.25


def test_zero_stays_zero_and_scale_does_not_matter():
    assert not ref.orthogonalize(np.zeros((3, 4))).any()
    g = np.random.default_rng(2).standard_normal((6, 9))
    np.testing.assert_allclose(ref.orthogonalize(1e4 * g), ref.orthogonalize(g), atol=1e-6)


def test_step():
    rng = np.random.default_rng(3)
    p, g, m = (rng.standard_normal((4, 6)) for _ in range(3))
    q, n, u = ref.step(p, g, m, lr=0.1, momentum=0.9, weight_decay=0.5, scale=0.5)
    np.testing.assert_allclose(n, 0.9 * m + 0.5 * g)
    np.testing.assert_allclose(u, 0.5 * g + 0.9 * n)
    np.testing.assert_allclose(q, 0.95 * p - 0.02 * np.sqrt(6) * ref.orthogonalize(u))
