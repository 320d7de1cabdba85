"""The gradients' norm at the ends of its range, against ``oracle.adamw32``."""

import numpy as np
import pytest
import torch

from oracle import adamw32 as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def bwd():
    from block_wise_dynamic_gb300 import build

    build.build()
    import block_wise_dynamic_gb300 as m

    return m


def draw(n, std, kind, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    return (torch.randn(n, generator=g, device=DEV, dtype=torch.float64) * std).to(TYPES[kind])


def check(bwd, grads, max_norm, loss_scale):
    factor, norm = bwd.GradNorm(grads).clip_scale(max_norm, loss_scale)
    rf, rn = ref.clip([t.double().cpu().numpy() for t in grads], max_norm, loss_scale)
    # squares and sums of up to 16 positive terms in fp32, halved by the root, then the norm's rounding and
    # the factor's four: 16 half units are more than either
    np.testing.assert_allclose(float(norm), rn, rtol=16 * 2.0 ** -24)
    np.testing.assert_allclose(float(factor), rf, rtol=16 * 2.0 ** -24)


# squares that pass fp32's range, are subnormal there, or vanish; 1e-18 to
# 1e-20 lie around the sums that fp32 still holds in full
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("std", [1e20, 3e18, 1e-17, 1e-18, 3e-19, 1e-19, 1e-20, 1e-24, 1e-37])
def test_ends_of_the_range(bwd, std, kind):
    grads = [draw(70001, std, kind, 1), draw(5, std, kind, 2)]
    check(bwd, grads, std, 1.0)
    check(bwd, [g[1:] for g in grads], std, 1.0)  # pieces of the first and last 16 bytes


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("mix", [(1e20, 1e-2), (1e-24, 1e-2), (1e20, 1e-24), (1e-24, 0.0)])
def test_mixed_sizes(bwd, mix, kind):
    grads = [draw(40000, std, kind, 3 + i) for i, std in enumerate(mix)]
    both = draw(9000, mix[0], kind, 7)
    both[::3] = draw(3000, mix[1], kind, 8)  # neighbours in one thread's pieces
    check(bwd, grads + [both], 1.0, 1.0)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_large_loss_scale(bwd, kind):
    """The scaled gradients' squares pass fp32's range, the norm is an ordinary number."""
    check(bwd, [draw(50000, 1e20, kind, 9)], 1.0, 2.0 ** 66)
    check(bwd, [draw(50000, 1e-24, kind, 9)], 1.0, 2.0 ** -80)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_step_with_a_large_gradient_is_taken(bwd, kind):
    p = torch.nn.Parameter(torch.ones(3000, dtype=TYPES[kind], device=DEV))
    p.grad = draw(3000, 1e20, kind, 10)
    opt = bwd.AdamW8bit([p], lr=0.5, state_bits=32)
    opt.step(grad_scale=opt.clip_scale(1.0)[0])
    assert torch.isfinite(p).all() and not torch.equal(p, torch.ones_like(p))


def test_zeros(bwd):
    g = torch.zeros(100_003, device=DEV)
    g[1::2] = -0.0
    factor, norm = bwd.GradNorm([g, g.bfloat16()]).clip_scale(1.0)
    assert float(norm) == 0.0 and float(factor) == 1.0
