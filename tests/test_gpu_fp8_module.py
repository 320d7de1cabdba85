"""``Fp8Linear`` in autograd: what it saves, what it computes and what it refuses."""

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def fp8():
    from block_wise_dynamic_gb300 import build

    build.build()
    from block_wise_dynamic_gb300 import fp8 as m

    return m


def make(fp8, rows, seed=1, n=200, k=300):
    torch.manual_seed(seed)
    layer = fp8.Fp8Linear(k, n, device=DEV)
    x = torch.randn(rows, k, device=DEV, dtype=torch.bfloat16).requires_grad_()
    return layer, x


def gradients(layer, x, dy):
    layer.zero_grad()
    x.grad = None
    layer(x).backward(dy)
    return [x.grad.clone(), layer.weight.grad.clone(), layer.bias.grad.clone()]


@pytest.mark.parametrize("rows", [5, 300])
def test_second_derivatives_are_refused(fp8, rows):
    layer, x = make(fp8, rows)
    y = layer(x)
    (dx,) = torch.autograd.grad(y.float().square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        (y.float().sum() + dx.float().square().sum()).backward()
    # dy that takes no gradient itself: dx still depends on the weight
    (dx,) = torch.autograd.grad(layer(x).float().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        (layer.bias.float().sum() + dx.float().square().sum()).backward()


@pytest.mark.parametrize("rows", [5, 300])
def test_first_derivatives_with_create_graph(fp8, rows):
    layer, x = make(fp8, rows)
    dy = torch.randn(rows, 200, device=DEV, dtype=torch.bfloat16)
    want = gradients(layer, x, dy)
    got = torch.autograd.grad(layer(x), [x, layer.weight, layer.bias], dy, create_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_the_mark_of_gradients_names_the_layer(fp8):
    layer, x = make(fp8, 20)
    loss = layer(x).float().square().sum()
    loss.backward(create_graph=True)  # some optimizers ask for it and use first derivatives only
    with pytest.raises(RuntimeError, match="Fp8Linear has no second derivatives"):
        x.grad.float().sum().backward()
