"""A copied or unpickled optimizer goes on as the original does."""

import copy
import io

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def by_pickle(x):
    f = io.BytesIO()
    torch.save(x, f)
    f.seek(0)
    return torch.load(f, weights_only=False)


@pytest.mark.parametrize("with_factor", [False, True])
@pytest.mark.parametrize("how", [copy.deepcopy, by_pickle])
def test_copies(how, with_factor):
    from block_wise_dynamic_gb300 import build

    build.build()
    import block_wise_dynamic_gb300 as bwd

    def step(opt, t):
        ps = [p for g in opt.param_groups for p in g["params"]]
        for p in ps:
            p.grad = torch.randn(p.shape, generator=torch.Generator(DEV).manual_seed(t), device=DEV)
        opt.step(grad_scale=opt.clip_scale(0.5)[0] if with_factor else None)
        return ps

    a = torch.nn.Parameter(torch.linspace(-1, 1, 5000, device=DEV))
    b = torch.nn.Parameter(torch.linspace(-1, 1, 300, device=DEV))
    opt = bwd.AdamW8bit([{"params": [a]}, {"params": [b], "state_bits": 32}], lr=1e-2)
    step(opt, 1)
    other = how(opt)
    for t in (2, 3):
        for p, q in zip(step(opt, t), step(other, t)):
            assert p is not q and torch.equal(p, q)
            for k, v in opt.state[p].items():
                assert int(v) == int(other.state[q][k]) == t if k == "step" else torch.equal(v, other.state[q][k])
