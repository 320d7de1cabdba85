"""A parameter group's ``state_bits`` is checked wherever a group comes from."""

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_groups_added_later():
    from block_wise_dynamic_gb300 import build

    build.build()
    import block_wise_dynamic_gb300 as bwd

    a, b = (torch.nn.Parameter(torch.ones(3000, device=DEV)) for _ in range(2))
    opt = bwd.AdamW8bit([a])
    for bits in (16, 0, None, "8"):
        with pytest.raises(ValueError):
            opt.add_param_group({"params": [b], "state_bits": bits})
    assert len(opt.param_groups) == 1
    opt.add_param_group({"params": [b], "state_bits": 32})
    a.grad, b.grad = torch.ones_like(a), torch.ones_like(b)
    opt.step()
    assert "m_codes" in opt.state[a] and "exp_avg" in opt.state[b]
    with pytest.raises(ValueError):
        bwd.AdamW8bit([{"params": [a]}, {"params": [b], "state_bits": 4}])
