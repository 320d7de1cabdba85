"""The 8-bit floating point layers, the mixed 8- and 32-bit optimizer and the
device-held gradient factor together."""

import copy

import numpy as np
import pytest
import torch

from oracle import adamw32 as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def bwd():
    from block_wise_dynamic_gb300 import build

    build.build()
    import block_wise_dynamic_gb300 as m

    m.init(0)
    return m


def state8(bwd, n, seed):
    """A state some steps old."""
    p = torch.randn(n, generator=torch.Generator(DEV).manual_seed(seed), device=DEV) * 0.02
    st = bwd.state_init(n, DEV)
    for t in (1, 2):
        g = torch.randn(n, generator=torch.Generator(DEV).manual_seed(seed + t), device=DEV) * 1e-3
        bwd.adam8bit_step_multi([p], [g], *[[x] for x in st], step=t)
    return p, st


@pytest.mark.parametrize("pk", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("gk", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n", [5, 2048, 3 * 2048 + 17, 70001])
def test_scaled_8bit_step_is_the_step_on_scaled_gradients(bwd, n, gk, pk):
    p, st = state8(bwd, n, 1)
    g = (torch.randn(n, generator=torch.Generator(DEV).manual_seed(9), device=DEV) * 1e-2).to(gk)
    factor = torch.full((1,), 0.37, device=DEV)
    a = [p.to(pk), *[x.clone() for x in st]]
    b = [p.to(pk), *[x.clone() for x in st]]
    bwd.MultiTensorArgs([a[0]], [g], *[[x] for x in a[1:]]).step(step=3, weight_decay=0.01, grad_scale=factor)
    bwd.MultiTensorArgs([b[0]], [g.float() * factor], *[[x] for x in b[1:]]).step(step=3, weight_decay=0.01)
    for x, y in zip(a[1:], b[1:]):
        assert torch.equal(x, y)
    # the same operations on the same numbers
    assert torch.equal(a[0], b[0])
    kept = [x.clone() for x in a]
    for bad in (float("nan"), float("inf")):
        factor.fill_(bad)
        bwd.MultiTensorArgs([a[0]], [g], *[[x] for x in a[1:]]).step(step=4, grad_scale=factor)
    assert all(torch.equal(x, y) for x, y in zip(a, kept))


def test_scaled_step_refusals(bwd):
    p, st = state8(bwd, 10, 2)
    args = bwd.MultiTensorArgs([p], [p.clone()], *[[x] for x in st])
    with pytest.raises(TypeError):
        args.step(step=3, grad_scale=torch.ones(1, device=DEV, dtype=torch.float16))
    with pytest.raises(ValueError):
        args.step(step=3, grad_scale=torch.ones(1))
    with pytest.raises(ValueError):
        bwd.AdamW8bit([torch.nn.Parameter(p)], state_bits=16)
    with pytest.raises(ValueError):
        bwd.AdamW8bit([torch.nn.Parameter(p)]).clip_scale(1.0)


def make(dtype):
    g = torch.Generator(DEV).manual_seed(5)
    return [torch.nn.Parameter((torch.randn(s, generator=g, device=DEV) * 0.02).to(dtype)) for s in ((40, 70), (33,), (5000,))]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_mixed_optimizer(bwd, dtype):
    """The 32-bit group follows the formula, the 8-bit one the optimizer
    without the other group."""
    ps, qs = make(dtype), make(dtype)
    opt = bwd.AdamW8bit([{"params": ps[:1]}, {"params": ps[1:], "state_bits": 32}], lr=1e-2, weight_decay=0.05)
    only = bwd.AdamW8bit(qs[:1], lr=1e-2, weight_decay=0.05)
    want = [(p.detach().double().cpu().numpy(), np.zeros(p.numel()), np.zeros(p.numel())) for p in ps[1:]]
    unit = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    for t in range(1, 5):
        for p in ps:
            p.grad = (torch.randn(p.shape, generator=torch.Generator(DEV).manual_seed(t), device=DEV) * 1e-2).to(dtype)
        qs[0].grad = ps[0].grad.clone()
        opt.step()
        only.step()
        before = [w[0] for w in want]
        for i, p in enumerate(ps[1:]):
            g = p.grad.double().cpu().numpy()
            want[i] = ref.step(*[want[i][0], g, *want[i][1:]], lr=1e-2, weight_decay=0.05, step=t)
            got = p.detach().double().cpu().numpy()
            # each step: p's rounding, and fp32 rounding of the update (at most lr, times the quotient's ten roundings)
            assert np.all(np.abs(got - want[i][0]) <= t * (2 * unit * np.abs(before[i]) + 2 * unit * 1e-2 + 1e-2 * 40 * 2.0 ** -24))
    assert torch.equal(ps[0], qs[0]) and torch.equal(opt.state[ps[0]]["m_codes"], only.state[qs[0]]["m_codes"])
    assert opt.state[ps[1]]["exp_avg"].dtype == torch.float32 and "m_codes" not in opt.state[ps[1]]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_resume_is_bit_exact(bwd, dtype):
    def build(ps):
        return bwd.AdamW8bit([{"params": ps[:1]}, {"params": ps[1:], "state_bits": 32}], lr=1e-2)

    def grads(ps, t):
        for p in ps:
            p.grad = (torch.randn(p.shape, generator=torch.Generator(DEV).manual_seed(t), device=DEV) * 1e-2).to(dtype)

    ps = make(dtype)
    opt = build(ps)
    for t in (1, 2):
        grads(ps, t)
        opt.step()
    saved = copy.deepcopy(opt.state_dict())
    qs = [torch.nn.Parameter(p.detach().clone()) for p in ps]
    again = build(qs)
    again.load_state_dict(saved)
    for t in (3, 4):
        grads(ps, t)
        grads(qs, t)
        opt.step()
        again.step()
    for p, q in zip(ps, qs):
        assert torch.equal(p, q)
        for k, v in opt.state[p].items():
            assert v == again.state[q][k] if k == "step" else torch.equal(v, again.state[q][k])


def test_clip_scale_over_groups_and_types(bwd):
    ps = make(torch.float32)[:1] + make(torch.bfloat16)[1:]
    for p in ps:
        p.grad = torch.randn_like(p)
    opt = bwd.Adam8bit([{"params": ps[:1]}, {"params": ps[1:], "state_bits": 32}])
    for scale in (1.0, 3.0):
        for p in ps:
            p.grad = p.grad * scale  # new tensors in the same places
        factor, norm = opt.clip_scale(0.5, 2.0)
        rf, rn = ref.clip([p.grad.double().cpu().numpy() for p in ps], 0.5, 2.0)
        np.testing.assert_allclose([float(factor), float(norm)], [rf, rn], rtol=1e-6)
    ps[0].grad[0, 0] = float("inf")
    before = [p.detach().clone() for p in ps]
    opt.step(grad_scale=opt.clip_scale(0.5)[0])
    assert all(torch.equal(a, b) for a, b in zip(before, ps))


def test_codec_keeps_fp32_groups(bwd):
    from block_wise_dynamic_gb300 import codec

    ps = make(torch.float32)
    full = torch.optim.AdamW(ps, lr=1e-3)
    for p in ps:
        p.grad = torch.randn_like(p)
    full.step()
    opt = bwd.AdamW8bit([{"params": ps[:1]}, {"params": ps[1:], "state_bits": 32}])
    codec.load_from_fp32_adam(opt, full)
    opt.step()
    out = codec.export_fp32_adam_state(opt)
    assert out[ps[1]]["exp_avg"].shape == ps[1].shape and float(out[ps[1]]["step"]) == 2.0
    m, _, _ = opt.state[ps[1]]["exp_avg"], None, None
    want = 0.9 * full.state[ps[1]]["exp_avg"].double() + 0.1 * ps[1].grad.double()
    np.testing.assert_allclose(m.double().cpu().numpy(), want.view(-1).cpu().numpy(), rtol=4 * 2.0 ** -24, atol=1e-7)


def test_the_demo_learns(bwd):
    """The text is predictable three times in four; chance is ln 512 = 6.24
    and the noise floor ln 4 + (1/4) ln 512 at most."""
    from block_wise_dynamic_gb300 import demo

    losses = demo.train(steps=120)
    assert losses[0] > 5.5 and all(np.isfinite(losses))
    assert np.mean(losses[-10:]) < np.log(4) + 0.25 * np.log(512) + 0.5
    bwd.check_device(0)
