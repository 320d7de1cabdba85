"""Every form of the 8-bit step takes the device-held factor and count."""

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def bwd():
    from block_wise_dynamic_gb300 import build

    build.build()
    import block_wise_dynamic_gb300 as m

    m.init(0)
    return m


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_one_tensor_and_a_list(bwd, dtype):
    n = 5000
    g = torch.linspace(-1, 1, n, device=DEV).to(dtype)
    factor = torch.full((1,), 0.5, device=DEV)
    results = []
    for how in range(4):
        p, st = torch.linspace(-2, 1, n, device=DEV).to(dtype), bwd.state_init(n, DEV)
        for t in (1, 2):
            if how == 0:
                bwd.MultiTensorArgs([p], [g], *[[x] for x in st]).step(step=t, grad_scale=factor)
            elif how == 1:
                bwd.adam8bit_step(p, g, *st, step=t, grad_scale=factor)
            elif how == 2:
                bwd.adam8bit_step_multi([p], [g], *[[x] for x in st], step=t, grad_scale=factor)
            else:
                bwd.adam8bit_step(p, g, *st, step=bwd.StepCount(DEV, t - 1), grad_scale=factor)
        results.append((p, *st))
    for r in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, results[0]))


def test_one_count_over_several_calls(bwd):
    p, st = torch.ones(3000, device=DEV), bwd.state_init(3000, DEV)
    m, v = torch.zeros(3000, device=DEV), torch.zeros(3000, device=DEV)
    count, count32 = bwd.StepCount(DEV), bwd.StepCount(DEV, 7)
    for f in (1.0, float("nan"), 1.0):
        scale = torch.full((1,), f, device=DEV)
        bwd.adam8bit_step(p, torch.ones_like(p), *st, step=count, grad_scale=scale)
        bwd.adam32_step_multi([p], [torch.ones_like(p)], [m], [v], step=count32, grad_scale=scale)
    assert int(count.taken) == 2 and int(count32.taken) == 9
    for call in (lambda c: bwd.adam8bit_step(p, torch.ones_like(p), *st, step=c),
                 lambda c: bwd.adam32_step_multi([p], [torch.ones_like(p)], [m], [v], step=c)):
        with pytest.raises(ValueError):
            call(bwd.StepCount("cpu"))
        with pytest.raises(bwd.BwdError):
            call(0)
