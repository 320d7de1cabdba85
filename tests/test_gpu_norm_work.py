"""``bwd_grad_norm`` keeps to the workspace that it asks for."""

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("count", [0, 1, 3, 1024, 1025, 2500])
@pytest.mark.parametrize("size", [1, 3000])
def test_nothing_beside_the_workspace_is_written(count, size):
    from block_wise_dynamic_gb300 import build

    build.build()
    import block_wise_dynamic_gb300 as bwd

    handle = bwd.GradNorm([torch.full((size,), 0.5, device=DEV) for _ in range(count)], device=DEV)
    work = bwd._lib.bwd_grad_norm_work_bytes(count)
    whole = torch.full((256 + work + 256,), 0xA5, dtype=torch.uint8, device=DEV)
    whole[256:256 + work] = 0
    handle._work = whole[256:256 + work]
    for _ in range(3):
        factor, norm = handle.clip_scale(1e9)
    assert float(norm) == pytest.approx(0.5 * (count * size) ** 0.5, rel=1e-6) and float(factor) == 1.0
    assert bool((whole[:256] == 0xA5).all()) and bool((whole[256 + work:] == 0xA5).all())
    assert not whole[256:272].any()
