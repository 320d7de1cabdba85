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


def test_gradients_may_be_changed_in_place():
    """As optimizers and clipping do with gradients made with create_graph."""
    from block_wise_dynamic_gb300._once import first_order

    class Scale(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, y):
            return 2 * x + 3 * y

        @staticmethod
        @first_order("Scale")
        def backward(ctx, dy):
            return 2 * dy, 3 * dy

    x, y = (torch.ones(2, requires_grad=True) for _ in range(2))
    dx, dy = torch.autograd.grad(Scale.apply(x, y).sum(), [x, y], create_graph=True)
    dx.mul_(2)
    with torch.no_grad():
        dy.add_(1)
    assert dx.tolist() == [4.0, 4.0] and dy.tolist() == [4.0, 4.0]
    for g in (dx, dy):
        with pytest.raises(RuntimeError, match="Scale has no second derivatives"):
            g.sum().backward()
