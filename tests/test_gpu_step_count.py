"""Steps whose factor is not finite write nothing and are not counted: the
bias corrections belong to the steps that the moments have seen."""

import copy

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


def make(dtype, grad_dtype=None):
    g = torch.Generator(DEV).manual_seed(5)
    ps = [torch.nn.Parameter((torch.randn(s, generator=g, device=DEV) * 0.02).to(dtype)) for s in ((40, 70), (33,), (5000,))]
    gradients(ps, 0)
    return ps


def gradients(ps, t):
    for p in ps:
        g = torch.randn(p.shape, generator=torch.Generator(DEV).manual_seed(t), device=DEV) * 1e-2
        p.grad = g.to(p.dtype)


def build(bwd, ps, split=True):
    groups = [{"params": ps[:1]}, {"params": ps[1:], "state_bits": 32}]
    return bwd.AdamW8bit(groups, lr=1e-2, weight_decay=0.05)


def factor(x):
    return torch.full((1,), x, device=DEV)


def same(a, b, ps, qs):
    for p, q in zip(ps, qs):
        assert torch.equal(p, q)
        for k, v in a.state[p].items():
            assert int(v) == int(b.state[q][k]) if k == "step" else torch.equal(v, b.state[q][k])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_skipped_steps_are_not_counted(bwd, dtype):
    ps, qs = make(dtype), make(dtype)
    opt, only = build(bwd, ps), build(bwd, qs)
    kept = [p.detach().clone() for p in ps]
    for t in range(10):
        opt.step(grad_scale=factor(float("nan") if t % 2 else float("inf")))
    assert all(torch.equal(p, k) for p, k in zip(ps, kept))
    assert all(int(opt.state[p]["step"]) == 0 for p in ps)
    for t in (1, 2, 3):
        gradients(ps, t)
        gradients(qs, t)
        opt.step(grad_scale=factor(0.5))
        opt.step(grad_scale=factor(float("nan")))
        only.step(grad_scale=factor(0.5))
        same(opt, only, ps, qs)
    assert all(int(opt.state[p]["step"]) == 3 for p in ps)


def test_first_step_after_skipped_ones_against_the_formula(bwd):
    p = torch.nn.Parameter(torch.linspace(-1, 1, 4001, device=DEV))
    p.grad = torch.linspace(-1e-2, 2e-2, 4001, device=DEV)
    opt = bwd.AdamW8bit([p], lr=1e-2, weight_decay=0.05, state_bits=32)
    old = p.detach().double().cpu().numpy()
    for _ in range(10):
        opt.step(grad_scale=factor(float("nan")))
    opt.step(grad_scale=factor(0.5))
    zero = old * 0
    want, m, v = ref.step(old, p.grad.double().cpu().numpy(), zero, zero, lr=1e-2, weight_decay=0.05, step=1, scale=0.5)
    # p's rounding, and the fp32 roundings of an update of at most lr (sixteen for the quotient and its scalars)
    assert abs(p.detach().double().cpu().numpy() - want).max() <= 2 * 2.0 ** -24 * 1.01 + 16 * 2.0 ** -24 * 1e-2


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_steps_with_and_without_a_factor_share_the_count(bwd, dtype):
    ps, qs = make(dtype), make(dtype)
    opt, only = build(bwd, ps), build(bwd, qs)
    for t, f in enumerate([None, 1.0, None, float("nan"), 1.0, None], 1):
        gradients(ps, t)
        gradients(qs, t)
        opt.step(grad_scale=None if f is None else factor(f))
        if f is None or f == 1.0:
            only.step()
    same(opt, only, ps, qs)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_parameter_that_joins_later_counts_its_own_steps(bwd, dtype):
    ps, qs = make(dtype), make(dtype)
    opt, only = build(bwd, ps), build(bwd, qs)
    for t, f in enumerate([1.0, float("nan"), 1.0, 1.0], 1):
        for xs in (ps, qs):
            gradients(xs, t)
            if t <= 2:
                xs[2].grad = None
        opt.step(grad_scale=factor(f))
        if f == 1.0:
            only.step()
    same(opt, only, ps, qs)
    assert [int(opt.state[p]["step"]) for p in ps] == [3, 3, 2]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_resume_keeps_the_count(bwd, dtype):
    ps = make(dtype)
    opt = build(bwd, ps)
    for f in (float("nan"), 1.0, float("nan"), 1.0):
        opt.step(grad_scale=factor(f))
    saved = copy.deepcopy(opt.state_dict())
    assert all(s["step"] == 2 and isinstance(s["step"], int) for s in saved["state"].values())
    live = opt.state_dict()
    qs = [torch.nn.Parameter(p.detach().clone()) for p in ps]
    again = build(bwd, qs)
    again.load_state_dict(saved)
    for t, f in ((3, 1.0), (4, float("nan")), (5, None)):
        gradients(ps, t)
        gradients(qs, t)
        for o in (opt, again):
            o.step(grad_scale=None if f is None else factor(f))
    same(opt, again, ps, qs)
    assert all(s["step"] == 2 for s in live["state"].values())


def test_codec_reads_the_count(bwd):
    from block_wise_dynamic_gb300 import codec

    ps = make(torch.float32)
    opt = build(bwd, ps)
    for f in (float("nan"), 1.0, 1.0):
        opt.step(grad_scale=factor(f))
    assert all(float(s["step"]) == 2.0 for s in codec.export_fp32_adam_state(opt).values())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_captured_step_replays_as_the_next_one(bwd, dtype):
    ps, qs = make(dtype), make(dtype)
    opt, eager = build(bwd, ps), build(bwd, qs)
    f = factor(0.5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        opt.step(grad_scale=f)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step(grad_scale=f)
    for x in (0.5, float("inf"), 0.25, 0.5):
        f.fill_(x)
        graph.replay()
    for x in (0.5, 0.5, 0.25, 0.5):
        eager.step(grad_scale=factor(x))
    torch.cuda.synchronize()
    same(opt, eager, ps, qs)
    assert all(int(opt.state[p]["step"]) == 4 for p in ps)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_captured_clipping_and_step(bwd, dtype):
    ps, qs = make(dtype), make(dtype)
    opt, eager = build(bwd, ps), build(bwd, qs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        opt.step(grad_scale=opt.clip_scale(0.1)[0])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        factor, norm = opt.clip_scale(0.1)
        opt.step(grad_scale=factor)
    eager.step(grad_scale=eager.clip_scale(0.1)[0])
    for t in (1, 2, 3):
        for p, q in zip(ps, qs):
            g = torch.randn(p.shape, generator=torch.Generator(DEV).manual_seed(t), device=DEV) * (float("nan") if t == 2 else 1e-2)
            p.grad.copy_(g)
            q.grad.copy_(g)
        graph.replay()
        eager.step(grad_scale=eager.clip_scale(0.1)[0])
    torch.cuda.synchronize()
    same(opt, eager, ps, qs)
    assert all(int(opt.state[p]["step"]) == 3 for p in ps)
