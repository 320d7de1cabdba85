"""Functions marked as having first derivatives only, on the CPU."""

import pytest
import torch


@pytest.fixture(scope="module")
def cube():
    from block_wise_dynamic_gb300._once import first_order

    class Cube(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, other):
            ctx.save_for_backward(x)
            return x ** 3

        @staticmethod
        @first_order("Cube")
        def backward(ctx, dy):
            (x,) = ctx.saved_tensors
            return dy * 3 * x ** 2, None

    return lambda x: Cube.apply(x, 1.0)


def test_first_derivatives(cube):
    x = torch.tensor([1.0, 2.0], requires_grad=True)
    cube(x).sum().backward()
    assert x.grad.tolist() == [3.0, 12.0] and not x.grad.requires_grad
    (dx,) = torch.autograd.grad(cube(x).sum(), x, create_graph=True)
    assert dx.tolist() == [3.0, 12.0]


@pytest.mark.parametrize("loss_depends_on_x_otherwise", [False, True])
@pytest.mark.parametrize("dy_takes_a_gradient", [False, True])
def test_second_derivatives_raise(cube, dy_takes_a_gradient, loss_depends_on_x_otherwise):
    x = torch.tensor([1.0, 2.0], requires_grad=True)
    y = cube(x)
    (dx,) = torch.autograd.grad((y * y if dy_takes_a_gradient else y).sum(), x, create_graph=True)
    loss = dx.square().sum() + (x.sum() if loss_depends_on_x_otherwise else 0.0)
    with pytest.raises(RuntimeError, match="Cube has no second derivatives"):
        loss.backward()
