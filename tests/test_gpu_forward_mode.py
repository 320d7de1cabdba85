"""Layers without forward-mode derivatives refuse them, with gradients switched off too."""

import pytest
import torch
from torch.autograd import forward_ad

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_wise_dynamic_gb300 import build

    build.build()


def layers():
    from block_wise_dynamic_gb300 import fp4, fp8, norm

    return {"norm": norm.LayerNorm(64), "fp8": fp8.Fp8Linear(64, 48, dtype=torch.float32), "fp4": fp4.Fp4Linear(torch.nn.Linear(64, 48, device=DEV))}


@pytest.mark.parametrize("name", ["norm", "fp8", "fp4"])
@pytest.mark.parametrize("grad", [True, False])
def test_a_tangent_is_refused(name, grad):
    layer, x = layers()[name], torch.randn(5, 64, device=DEV)
    with torch.no_grad():
        want = layer(x)
    with torch.set_grad_enabled(grad), forward_ad.dual_level():
        with pytest.raises(RuntimeError):
            layer(forward_ad.make_dual(x, torch.ones_like(x)))
        # without one, inside a level too, it is as ever
        assert torch.equal(layer(x).detach(), want)
    with torch.set_grad_enabled(grad), pytest.raises(RuntimeError):
        torch.func.jvp(layer, (x,), (torch.ones_like(x),))


@pytest.mark.parametrize("name", ["norm", "fp8"])
def test_a_weights_tangent_is_refused(name):
    layer, x = layers()[name], torch.randn(5, 64, device=DEV)
    weight = layer.weight.detach()
    with torch.no_grad(), forward_ad.dual_level():
        del layer.weight
        layer.weight = forward_ad.make_dual(weight, torch.ones_like(weight))
        with pytest.raises(RuntimeError):
            layer(x)
