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


@pytest.mark.parametrize("rows", [5, 300])
def test_saved_tensor_hooks_see_the_codes(fp8, rows):
    """What a hook gives back, at another address, is what backward reads."""
    layer, x = make(fp8, rows)
    dy = torch.randn(rows, 200, device=DEV, dtype=torch.bfloat16)
    want = gradients(layer, x, dy)
    sizes = []

    def pack(t):
        sizes.append(t.numel() * t.element_size())
        return t.cpu()

    with torch.autograd.graph.saved_tensors_hooks(pack, lambda t: t.to(DEV)):
        got = gradients(layer, x, dy)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert sum(sizes) >= rows * 300 + 200 * 300


def test_checkpointing(fp8):
    from torch.utils.checkpoint import checkpoint

    layer, x = make(fp8, 700)
    dy = torch.randn(700, 200, device=DEV, dtype=torch.bfloat16)
    want = gradients(layer, x, dy)
    layer.zero_grad()
    x.grad = None
    checkpoint(layer, x, use_reentrant=False).backward(dy)
    assert all(torch.equal(a, b) for a, b in zip([x.grad, layer.weight.grad, layer.bias.grad], want))


def test_backward_frees_what_forward_saved(fp8):
    rows, n, k = 2048, 1024, 4096
    layer, x = make(fp8, rows, n=n, k=k)
    x.grad, layer.weight.grad, layer.bias.grad = torch.zeros_like(x), torch.zeros_like(layer.weight), torch.zeros_like(layer.bias)
    y = layer(x)
    held = torch.cuda.memory_allocated()
    y.backward(torch.zeros_like(y))
    assert held - torch.cuda.memory_allocated() >= rows * k + n * k  # y and its graph are still there
    with pytest.raises(RuntimeError):
        y.backward(torch.zeros_like(y))


@pytest.mark.parametrize("rows", [5, 300])
def test_hooks_may_give_back_any_place(fp8, rows):
    layer, x = make(fp8, rows)
    dy = torch.randn(rows, 200, device=DEV, dtype=torch.bfloat16)
    want = gradients(layer, x, dy)

    def unpack(t):
        other = torch.zeros(t.numel() + 5, dtype=t.dtype, device=DEV)[5:]
        return other.copy_(t)

    with torch.autograd.graph.saved_tensors_hooks(lambda t: t.clone(), unpack):
        got = gradients(layer, x, dy)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.fixture
def calls(fp8, monkeypatch):
    seen = []
    launch = fp8._launch

    def spy(entry, device, stream, *args):
        seen.append((entry, args))
        return launch(entry, device, stream, *args)

    monkeypatch.setattr(fp8, "_launch", spy)
    return seen


def column_codes(calls):
    """The column codes that bwd_fp8_linear was asked for, one for each call of it."""
    return [args[11] for entry, args in calls if entry == "bwd_fp8_linear"]


@pytest.mark.parametrize("rows", [1, 16, 300])
def test_only_a_weight_gradient_needs_column_codes(fp8, calls, rows):
    layer, x = make(fp8, rows)
    want = layer(x)
    assert column_codes(calls)[-1] is not None
    with torch.no_grad():
        y = layer(x)
    assert column_codes(calls)[-1] is None and torch.equal(y, want) and not y.requires_grad
    with torch.inference_mode():
        assert torch.equal(layer(x), want) and column_codes(calls)[-1] is None
    dy = torch.randn_like(want)
    dx = gradients(layer, x, dy)[0]
    layer.weight.requires_grad_(False)
    layer.weight.grad = layer.bias.grad = x.grad = None
    y = layer(x)
    assert column_codes(calls)[-1] is None and torch.equal(y, want)
    y.backward(dy)
    assert torch.equal(x.grad, dx) and layer.weight.grad is None and layer.bias.grad is not None
    layer.bias.requires_grad_(False)
    y = layer(x.detach())
    assert column_codes(calls)[-1] is None and torch.equal(y, want) and not y.requires_grad
