"""The 64-bit layer norm against torch's own and against differences."""

import numpy as np
import torch

from oracle import layer_norm as ref


def test_forward_and_backward_are_torchs():
    rng = np.random.default_rng(0)
    x, dy = rng.standard_normal((7, 13)) + 2.0, rng.standard_normal((7, 13))
    gamma, beta = rng.standard_normal(13), rng.standard_normal(13)
    t = [torch.tensor(a, requires_grad=True) for a in (x, gamma, beta)]
    y = torch.nn.functional.layer_norm(t[0], (13,), t[1], t[2], 1e-5)
    y.backward(torch.tensor(dy))
    got, mean, rstd = ref.forward(x, gamma, beta)
    np.testing.assert_allclose(got, y.detach().numpy(), rtol=1e-12, atol=1e-12)
    for a, b in zip(ref.backward(dy, x, gamma, mean, rstd), t):
        np.testing.assert_allclose(a, b.grad.numpy(), rtol=1e-11, atol=1e-11)


def test_backward_is_the_differences():
    rng = np.random.default_rng(1)
    x, dy, gamma, beta = (rng.standard_normal(s) for s in ((3, 5), (3, 5), 5, 5))
    _, mean, rstd = ref.forward(x, gamma, beta)
    grads = ref.backward(dy, x, gamma, mean, rstd)
    for i, (a, g) in enumerate(zip((x, gamma, beta), grads)):
        for at in np.ndindex(a.shape):
            sides = []
            for h in (1e-6, -1e-6):
                moved = [x.copy(), gamma.copy(), beta.copy()]
                moved[i][at] += h
                sides.append((ref.forward(*moved)[0] * dy).sum())
            assert abs((sides[0] - sides[1]) / 2e-6 - g[at]) < 1e-7
