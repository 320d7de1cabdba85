"""Kernels that begin before the kernel ahead of them has ended read what that one writes."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_wise_dynamic_gb300 import build

    build.build()


def values(rows, cols, seed, dtype):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal((rows, cols))).to(DEV, dtype)


def test_layers_behind_one_another():
    """Each call's input is the result of the one before, in memory that held another result a moment ago."""
    from block_wise_dynamic_gb300 import fp4, fp8, norm

    width = 512
    w = values(width, width, 1, torch.bfloat16) * width ** -0.5
    w4, w8 = fp4.quantize(w), fp8.quantize(w, "tiles")
    gamma = torch.ones(width, device=DEV)

    def chain(x, wait):
        for _ in range(8):
            for call in (lambda t: norm.forward(t, gamma)[0], lambda t: fp4.linear(t, w4), lambda t: norm.forward(t, gamma)[0],
                         lambda t: fp8.linear(t, w8)):
                x = call(x)
                if wait:
                    torch.cuda.synchronize()
        return x

    for rows in (1, 5, 40):
        starts = [values(rows, width, 10 + i, torch.bfloat16) for i in range(6)]
        want = [chain(x, True) for x in starts]
        for _ in range(3):
            got = [chain(x, False) for x in starts]
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_updates_behind_one_another():
    from block_wise_dynamic_gb300 import muon

    for shape in ((40, 70), (300, 200), (64, 1000)):
        gs = [values(*shape, 20 + i, torch.float32) for i in range(4)]
        want = []
        for g in gs:
            want.append(muon.orthogonalize(g))
            torch.cuda.synchronize()
        for _ in range(10):
            got = [muon.orthogonalize(g) for g in gs]
            assert all(torch.equal(a, b) for a, b in zip(got, want))
