"""What an optimizer's ``clip_scale`` returns stays what it was."""

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def bwd():
    from block_wise_dynamic_gb300 import build

    build.build()
    import block_wise_dynamic_gb300 as m

    return m


def test_later_calls_leave_earlier_results_alone(bwd):
    """A run that keeps each step's norm, without waiting for it, and reads them at the end."""
    p = torch.nn.Parameter(torch.zeros(1000, device=DEV))
    opt = bwd.AdamW8bit([p])
    kept = []
    for t in range(1, 5):
        p.grad = torch.full_like(p, float(t))
        kept.append(opt.clip_scale(2.0))
    for t, (factor, norm) in enumerate(kept, 1):
        want = t * 1000 ** 0.5
        assert float(norm) == pytest.approx(want, rel=1e-6) and float(factor) == pytest.approx(2.0 / want, rel=1e-6)
