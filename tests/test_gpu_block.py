"""Layer norm, orthogonalised updates and 4-bit layers together, as a model
uses them: a block is trained with the first two and served with the third."""

import numpy as np
import pytest
import torch

from oracle import fp4 as q4
from oracle import layer_norm as ln
from oracle import muon as ns

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def bwd():
    from block_wise_dynamic_gb300 import build

    build.build()
    import block_wise_dynamic_gb300 as m

    m.init(0)
    return m


def np64(t):
    return t.detach().double().cpu().numpy()


class Block(torch.nn.Module):
    def __init__(self, norm, dim, wide):
        super().__init__()
        torch.manual_seed(0)
        self.norm = norm.LayerNorm(dim)
        self.up = torch.nn.Linear(dim, wide, device=DEV)
        self.down = torch.nn.Linear(wide, dim, device=DEV)
        self.last = norm.LayerNorm(dim, bias=False)

    def forward(self, x):
        return self.last(x + self.down(torch.relu(self.up(self.norm(x)))))


def in64(block, x, dy):
    """The same block's output and gradients by torch's own operations in binary64."""
    copy = {k: v.detach().double().cpu().requires_grad_() for k, v in block.named_parameters()}
    x = x.detach().double().cpu().requires_grad_()
    f = torch.nn.functional
    h = f.layer_norm(x, x.shape[-1:], copy["norm.weight"], copy["norm.bias"], 1e-5)
    h = f.linear(torch.relu(f.linear(h, copy["up.weight"], copy["up.bias"])), copy["down.weight"], copy["down.bias"])
    y = f.layer_norm(x + h, x.shape[-1:], copy["last.weight"], None, 1e-5)
    y.backward(dy.double().cpu())
    return y, x.grad, {k: v.grad for k, v in copy.items()}


def test_a_block_in_training(bwd):
    from block_wise_dynamic_gb300 import norm

    block = Block(norm, 96, 250)
    g = torch.Generator(DEV).manual_seed(1)
    x = torch.randn(4, 33, 96, generator=g, device=DEV).requires_grad_()
    dy = torch.randn(4, 33, 96, generator=g, device=DEV)
    y = block(x)
    y.backward(dy)
    want_y, want_x, want = in64(block, x, dy)
    # sums of up to 250 and 132 terms in fp32, three operators deep: 1e-5 of a gradient's norm is some 160 roundings
    for got, w in [(y, want_y), (x.grad, want_x)] + [(p.grad, want[k]) for k, p in block.named_parameters()]:
        assert np.linalg.norm(np64(got) - w.detach().numpy()) <= 1e-5 * np.linalg.norm(w.detach().numpy())
    matrices = [block.up.weight, block.down.weight]
    vectors = [p for p in block.parameters() if p.dim() == 1]
    opts = bwd.Muon(matrices, lr=0.1), bwd.AdamW8bit(vectors, lr=1e-3, state_bits=32, weight_decay=0.0)
    before = [np64(p) for p in matrices]
    for opt in opts:
        factor, _ = opt.clip_scale(0.5)
        opt.step(grad_scale=factor)
        if opt is opts[0]:
            scale = float(factor)
    for p, b in zip(matrices, before):
        want_p = ns.step(b, np64(p.grad), 0 * b, lr=0.1, momentum=0.95, scale=scale)[0]
        # five steps stretch fp32 roundings by up to 4.3 each: 1e-4 of the update's norm
        assert np.linalg.norm(np64(p) - want_p) <= 1e-4 * np.linalg.norm(want_p - b)
    assert torch.isfinite(block(x)).all()
    bwd.check_device(0)


def test_a_block_in_service(bwd):
    from block_wise_dynamic_gb300 import fp4, norm

    block = Block(norm, 96, 250)
    up, down = fp4.Fp4Linear(block.up), fp4.Fp4Linear(block.down)
    for tokens in (1, 7, 40):
        x = torch.randn(tokens, 96, generator=torch.Generator(DEV).manual_seed(tokens), device=DEV)
        with torch.no_grad():
            h = block.norm(x)
            a = up(h)
            y = down(torch.relu(a))
        # each stage from the one before it as it is: quantizing is a step function
        want = ln.forward(np64(x), np64(block.norm.weight), np64(block.norm.bias))[0]
        assert np.abs(np64(h) - want).max() <= 1e-5 * np.abs(want).max()
        for got, src, layer in ((a, h, block.up), (y, torch.relu(a), block.down)):
            want, size = q4.linear(np64(src), np64(layer.weight), np64(layer.bias))
            assert (np.abs(np64(got) - want) <= 2.0 ** -19 * size).all()  # eight instructions' truncations of 2^-22


def test_training_and_serving_a_step_at_a_time_in_a_graph(bwd):
    """Norm, its gradients, the update and the 4-bit product captured together; replays are the eager calls."""
    from block_wise_dynamic_gb300 import fp4, muon, norm

    g = torch.Generator(DEV).manual_seed(3)
    x, dy = (torch.randn(50, 64, generator=g, device=DEV) for _ in range(2))
    gamma = torch.ones(64, device=DEV)

    def state():
        return [torch.randn(40, 64, generator=torch.Generator(DEV).manual_seed(4), device=DEV)], [torch.zeros(40, 64, device=DEV)]

    def work(p, grad, args):
        y, mean, rstd = norm.forward(x, gamma)
        dx, dgamma, _ = norm.backward(dy, x, gamma, mean, rstd)
        grad.copy_(dx[:40])
        args.step(lr=0.1)
        return y, dgamma, fp4.linear(y, fp4.quantize(p))

    results = []
    for captured in (False, True):
        p, m = state()
        grad = torch.zeros(40, 64, device=DEV)
        args = muon.MuonArgs(p, [grad], m)
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                out = work(p[0], grad, args)
            for _ in range(3):
                graph.replay()
        else:
            for _ in range(3):
                out = work(p[0], grad, args)
        torch.cuda.synchronize()
        results.append([t.clone() for t in (*out, p[0], m[0])])
    assert all(torch.equal(a, b) for a, b in zip(*results))


def test_the_demo_with_orthogonalised_updates(bwd):
    from block_wise_dynamic_gb300 import demo

    lines = []
    losses = demo.train(steps=8, vocab=64, dim=64, batch=256, muon=True, log=lines.append)
    assert len(losses) == 8 and all(np.isfinite(losses)) and "4-bit" in lines[-1]
    bwd.check_device(0)
