"""``StableEmbedding`` has first derivatives only, and says so."""

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_second_derivatives_are_refused():
    from block_wise_dynamic_gb300 import build

    build.build()
    from block_wise_dynamic_gb300.embedding import StableEmbedding

    layer = StableEmbedding(50, 64, device=DEV)
    ids = torch.tensor([3, 7, 3, 49], device=DEV)
    dy = torch.randn(4, 64, device=DEV)
    layer(ids).backward(dy)
    want = [p.grad.clone() for p in layer.parameters()]
    layer.zero_grad()
    got = torch.autograd.grad(layer(ids), list(layer.parameters()), dy, create_graph=True)
    assert all(torch.allclose(a, b) for a, b in zip(got, want))  # rows that occur twice are added atomically
    with pytest.raises(RuntimeError, match="StableEmbedding has no second derivatives"):
        (layer.weight.sum() + got[0].square().sum()).backward()
