"""Orthogonalised updates and the Muon step against the 64-bit statement."""

import copy

import numpy as np
import pytest
import torch

from oracle import muon as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
U = 2.0 ** -24
ROUND = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


@pytest.fixture(scope="module")
def muon():
    from block_wise_dynamic_gb300 import build

    build.build()
    from block_wise_dynamic_gb300 import muon as m

    return m


def np64(t):
    return t.detach().double().cpu().numpy()


def draw(rows, cols, seed, kind="gauss", dtype=torch.float32):
    rng = np.random.default_rng(seed)
    g = rng.standard_normal((rows, cols))
    if kind == "strong":  # a few directions far above the rest
        r = max(1, min(rows, cols) // 32)
        g = 0.02 * g + rng.standard_normal((rows, r)) @ rng.standard_normal((r, cols))
    return torch.from_numpy(1e-3 * g).to(DEV).to(dtype)


def error_bound(g, steps, dtype):
    """Frobenius norm of the error, before the result is rounded.

    F is X's Frobenius norm, its spectral norm is below 1.21.  An operand is
    off by d of its value, a product's sum by e of the sum of its terms'
    magnitudes: both operands' roundings (2 d), and what the matrix
    instruction's truncated additions lose, 2e-10 a term, three terms to a
    product of pairs.  In one step
      A       e F^2, times |b| + 2 c |A| and |X|: (4.8 + 6.0) 1.21 e F^2
      A A     e |A|_F^2 <= 1.47 e F^2, times c |X|: 3.7 e F^2
      B's rounding  d |B|_F |X| with |B|_F <= (4.8 + 3.0) 1.21 F: 11.5 d F
      A's rounding  d |A|_F, times as for A: 16 d F
      B X     e |B|_F F <= 9.5 e F^2
    in all 27 e F^2 + 28 d F, and X's own rounding d F after it.  Later steps
    stretch an error by up to 4.3, the largest slope of a s + b s^3 + c s^5 and
    of its divided differences for s up to 1.21.  Beside its relative rounding, what
    is stored (times 2^14) is off by half of fp16's least subnormal."""
    xs = ref.iterates(np64(g), steps)
    m, n = xs[0].shape
    least = 2.0 ** -39 * (m * n) ** 0.5
    total = 2.0 ** -20 * np.linalg.norm(xs[0]) + least  # normalised in fp32, then rounded
    for i, x in enumerate(xs[:-1]):
        single = dtype == torch.bfloat16 and i + 1 == steps
        d = 2.0 ** -11 if single else 2.0 ** -22 + 2.0 ** -30
        e = 2.02 * d + 2e-10 * (1 if single else 3) * n
        f = np.linalg.norm(x)
        total = 4.3 * total + 27 * e * f * f + 29 * d * f + 17.5 * least
    return total


def check(out, g, steps=5):
    assert out.shape == g.shape and out.dtype == g.dtype
    want = ref.orthogonalize(np64(g), steps)
    off = np.linalg.norm(np64(out) - want)
    bound = error_bound(g, steps, g.dtype)
    bound += ROUND[g.dtype] * (np.linalg.norm(want) + bound) + TINY[g.dtype] * want.size ** 0.5
    assert off <= bound, (off, bound)


SHAPES = [(1, 1), (1, 100), (2, 3), (16, 16), (64, 64), (65, 130), (100, 300), (128, 128), (255, 257), (256, 256), (257, 600), (300, 300),
          (33, 1000), (512, 700), (640, 641), (17, 5000)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", SHAPES)
def test_orthogonalize(muon, shape, dtype):
    for kind in ("gauss", "strong"):
        for rows, cols in {shape, shape[::-1]}:
            g = draw(rows, cols, 1, kind, TYPES[dtype])
            before = g.clone()
            check(muon.orthogonalize(g), g)
            assert torch.equal(g, before)


@pytest.mark.parametrize("steps", [1, 2, 7])
def test_steps(muon, steps):
    for dtype in (torch.float32, torch.bfloat16):
        g = draw(200, 333, 2, "strong", dtype)
        check(muon.orthogonalize(g, steps), g, steps)


def test_pairs_are_needed_and_used(muon):
    """The strong directions' roundings would show among the weak ones: far more than fp32 results may be off."""
    g = draw(256, 512, 3, "strong")
    want = ref.orthogonalize(np64(g))
    assert np.linalg.norm(np64(muon.orthogonalize(g)) - want) < 1e-4 * np.linalg.norm(want)


@pytest.mark.parametrize("shape", [(1000, 2100), (1500, 1100)])
def test_larger(muon, shape):
    """Several tiles in both directions, and both widths of them."""
    g = draw(*shape, 4, "strong")
    check(muon.orthogonalize(g), g)


def test_batches(muon):
    """More matrices than one launch takes.  (How a sum is divided depends on
    how many there are, and with it a result's last bits.)"""
    g = torch.stack([draw(40, 70, i, "strong") for i in range(140)]).view(2, 70, 40, 70)
    out = muon.orthogonalize(g)
    assert out.shape == g.shape
    for i, j in [(0, 0), (0, 63), (0, 64), (1, 0), (1, 69)]:
        check(out[i, j], g[i, j])
    assert torch.equal(muon.orthogonalize(g), out)
    # a transposed view, and one that starts off every boundary
    flat = torch.zeros(40 * 70 + 1, device=DEV)
    flat[1:] = g[0, 0].reshape(-1)
    assert torch.equal(muon.orthogonalize(flat[1:].view(40, 70)), muon.orthogonalize(g[0, 0]))
    check(muon.orthogonalize(g[0, 0].t()), g[0, 0].t())


def test_special_matrices(muon):
    g = torch.stack([draw(70, 90, i) for i in range(6)])
    want = muon.orthogonalize(g)
    g[1] = 0
    g[2, 3, 4] = float("nan")
    g[3, 0, 0] = float("inf")
    g[4] *= 1e30
    g[5] *= 1e-20
    out = muon.orthogonalize(g)
    assert torch.equal(out[0], want[0]) and not out[1].any()
    assert out[2].isnan().all() and out[3].isnan().all()
    check(out[4], g[4])
    check(out[5], g[5])
    # squares and norm beyond fp32's range
    big = draw(300, 300, 9) * 1e37
    big = big / big.abs().max() * 3e38
    check(muon.orthogonalize(big), big)


def test_nothing(muon):
    for shape in [(0, 5), (5, 0), (0, 3, 4)]:
        assert muon.orthogonalize(torch.empty(shape, device=DEV)).shape == shape


def lists(shapes, p_type, g_type, seed=0):
    ps = [draw(r, c, seed + i) * 20 for i, (r, c) in enumerate(shapes)]
    gs = [draw(r, c, seed + 100 + i, "strong") for i, (r, c) in enumerate(shapes)]
    ms = [draw(r, c, seed + 200 + i, "strong") * 3 for i, (r, c) in enumerate(shapes)]
    return [p.to(p_type) for p in ps], [g.to(g_type) for g in gs], ms


def check_step(before, after, scale=1.0, **hp):
    (p0, g, m0), (p1, m1) = before, after
    want_p, want_m, u = ref.step(np64(p0), np64(g), np64(m0), scale=scale, **hp)
    gs, ms = np.abs(scale * np64(g)), np.abs(hp["momentum"] * np64(m0))
    # s g and mu, which is an fp32 number there, each within U of its own, then one fused multiply and add
    assert (np.abs(np64(m1) - want_m) <= U * (gs + ms) + 1.01 * U * np.abs(want_m) + 2.0 ** -148).all()
    # the update's relative error from its own roundings, stretched by at most 4.3^steps
    kind = p0.dtype
    step = hp["lr"] * hp.get("rms", 0.2) * max(u.shape) ** 0.5
    grown = 4.3 ** hp.get("steps", 5) * 4 * U * np.linalg.norm(gs + ms + np.abs(want_m)) / (np.linalg.norm(u) + ref.EPS)
    off = step * (error_bound(torch.from_numpy(u), hp.get("steps", 5), kind) + grown) * (1 + 4 * U)
    off += 4 * U * (np.abs(np64(p0)) + np.abs(want_p))
    got = np64(p1)
    assert np.isfinite(got).all()
    assert (np.abs(got - want_p) <= off + ROUND[kind] * (np.abs(want_p) + off) + TINY[kind]).all()


SET = [(300, 200), (200, 300), (64, 100), (300, 200), (1, 50), (257, 31)]


@pytest.mark.parametrize("p_type,g_type", [("fp32", "fp32"), ("fp32", "bf16"), ("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp32")])
@pytest.mark.parametrize("nesterov", [True, False])
def test_step(muon, p_type, g_type, nesterov):
    ps, gs, ms = lists(SET, TYPES[p_type], TYPES[g_type])
    hp = dict(lr=0.02, momentum=0.95, nesterov=nesterov, weight_decay=0.1, rms=0.3, steps=4)
    args = muon.MuonArgs(ps, gs, ms)
    for scale in (None, 0.37):
        before = [(p.clone(), g.clone(), m.clone()) for p, g, m in zip(ps, gs, ms)]
        args.step(**hp, grad_scale=None if scale is None else torch.full((1,), scale, device=DEV))
        for b, p, m in zip(before, ps, ms):
            check_step(b, (p, m), 1.0 if scale is None else float(np.float32(scale)), **hp)
        assert all(torch.equal(b[1], g) for b, g in zip(before, gs))


def test_many_shapes_at_once(muon):
    """More shapes than one launch takes, more matrices than that, and large ones between them."""
    shapes = [(20 + 7 * i, 50 + 31 * (i % 5)) for i in range(19)] + [(700, 1900), (40, 30), (1900, 700)] + [(33, 65)] * 50 + [(1, 1)]
    ps, gs, ms = lists(shapes, torch.float32, torch.float32)
    before = [(p.clone(), g.clone(), m.clone()) for p, g, m in zip(ps, gs, ms)]
    hp = dict(lr=0.1, momentum=0.9)
    muon.MuonArgs(ps, gs, ms).step(**hp)
    for b, p, m in zip(before, ps, ms):
        check_step(b, (p, m), **hp)


def test_a_factor_that_is_not_finite_writes_nothing(muon):
    ps, gs, ms = lists(SET, torch.float32, torch.float32)
    before = [t.clone() for t in ps + ms]
    args = muon.MuonArgs(ps, gs, ms)
    for bad in (float("nan"), float("inf")):
        args.step(grad_scale=torch.full((1,), bad, device=DEV))
    assert all(torch.equal(a, b) for a, b in zip(before, ps + ms))


def test_matrices_without_gradient_stay(muon):
    ps, gs, ms = lists([(30, 40), (40, 30)], torch.float32, torch.float32)
    gs[1].zero_(), ms[1].zero_()
    before = ps[1].clone()
    muon.MuonArgs(ps, gs, ms).step()
    assert torch.equal(ps[1], before) and not ms[1].any()


def test_graph_replay_and_streams(muon):
    ps, gs, ms = lists(SET, torch.float32, torch.bfloat16)
    twin = [[t.clone() for t in l] for l in (ps, gs, ms)]
    args, other = muon.MuonArgs(ps, gs, ms), muon.MuonArgs(*twin)
    factor = torch.ones(1, device=DEV)
    args.step(grad_scale=factor), other.step(grad_scale=factor)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        args.step(grad_scale=factor)
    factor.fill_(0.5)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    other.step(grad_scale=factor, stream=side)
    other.step(grad_scale=factor, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ps + ms, twin[0] + twin[2]))
    g = draw(100, 60, 1)
    want = muon.orthogonalize(g)
    torch.cuda.synchronize()
    got = muon.orthogonalize(g, stream=side)
    side.synchronize()
    assert torch.equal(want, got)


def model(dtype=torch.float32):
    torch.manual_seed(0)
    return torch.nn.ModuleList([torch.nn.Linear(40, 60, bias=False), torch.nn.Conv2d(8, 12, 3, bias=False), torch.nn.Linear(60, 40, bias=False)]
                               ).to(DEV, dtype)


def give_gradients(m, seed):
    for i, p in enumerate(m.parameters()):
        p.grad = draw(p.shape[0], p[0].numel(), seed + i, "strong", p.dtype).view(p.shape)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_optimizer(muon, dtype):
    m = model(TYPES[dtype])
    opt = muon.Muon(m.parameters(), lr=0.05, weight_decay=0.01)
    mom = [torch.zeros(p.shape[0], p[0].numel(), device=DEV) for p in m.parameters()]
    for t in range(3):
        give_gradients(m, 10 * t)
        before = [p.detach().clone().view(p.shape[0], -1) for p in m.parameters()]
        factor, norm = opt.clip_scale(1e-2)
        opt.step(grad_scale=factor)
        for p, b, v in zip(m.parameters(), before, mom):
            new = opt.state[p]["momentum_buffer"].view(p.shape[0], -1)
            check_step((b, p.grad.view(p.shape[0], -1), v), (p.detach().view(p.shape[0], -1), new), float(factor), lr=0.05, momentum=0.95,
                       weight_decay=0.01)
            v.copy_(new)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_optimizer_resumes(muon, dtype):
    m = model(TYPES[dtype])
    opt = muon.Muon(m.parameters())
    give_gradients(m, 0)
    opt.step()
    saved, weights = copy.deepcopy(opt.state_dict()), copy.deepcopy(m.state_dict())
    other = copy.deepcopy(opt)
    give_gradients(m, 50)
    opt.step()
    m2 = model(TYPES[dtype])
    m2.load_state_dict(weights)
    opt2 = muon.Muon(m2.parameters())
    opt2.load_state_dict(saved)
    give_gradients(m2, 50)
    opt2.step()
    assert all(torch.equal(a, b) for a, b in zip(m.parameters(), m2.parameters()))
    assert other.state_dict()["state"].keys() == saved["state"].keys()


def test_optimizer_groups_and_missing_gradients(muon):
    m = model()
    ps = list(m.parameters())
    opt = muon.Muon([{"params": ps[:1], "lr": 0.5}, {"params": ps[1:]}])
    give_gradients(m, 0)
    ps[2].grad = None
    before = [p.detach().clone() for p in ps]
    opt.step()
    assert torch.equal(ps[2], before[2]) and not torch.equal(ps[1], before[1])
    with pytest.raises(ValueError, match="matrices"):
        opt.add_param_group({"params": [torch.nn.Parameter(torch.zeros(3, device=DEV))]})
    assert len(opt.param_groups) == 2
    give_gradients(m, 5)  # another set of gradients than the plan's
    opt.step()
    assert not torch.equal(ps[2], before[2])


def test_optimizer_refusals(muon):
    p = torch.nn.Parameter(torch.zeros(4, 6, device=DEV).t())
    p.grad = torch.ones(6, 4, device=DEV)
    with pytest.raises(ValueError, match="contiguous"):
        muon.Muon([p]).step()
    p = torch.nn.Parameter(torch.zeros(4, 6, device=DEV))
    opt = muon.Muon([p])
    with pytest.raises(ValueError, match="no parameter has a gradient"):
        opt.clip_scale(1.0)
    opt.step()  # nothing to do
    p.grad = torch.ones(4, 6, device=DEV)
    opt.step()
    p.grad = torch.ones(4, 6, device=DEV).t().contiguous().t()  # of another layout: copied
    opt.step()
    assert torch.isfinite(p).all()
    opt.param_groups[0]["lr"] = -1.0
    from block_wise_dynamic_gb300 import BwdError

    before = p.detach().clone()
    with pytest.raises(BwdError):
        opt.step()
    assert torch.equal(p, before)


def test_two_streams_at_once(muon):
    """Lists with workspaces of their own, small and large matrices, side by side."""
    sets = [lists([(300, 200), (64, 100)], torch.float32, torch.float32, s) for s in (0, 1000)]
    sets += [lists([(700, 1900)], torch.float32, torch.float32, 2000)]
    alone = [[[t.clone() for t in l] for l in s] for s in sets]
    for s in alone:
        args = muon.MuonArgs(*s)
        for _ in range(5):
            args.step()
    args = [muon.MuonArgs(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        for a, st in zip(args, streams):
            a.step(stream=st)
    torch.cuda.synchronize()
    for s, t in zip(sets, alone):
        assert all(torch.equal(a, b) for a, b in zip(s[0] + s[2], t[0] + t[2]))


def test_fifty_thousand_columns(muon):
    """A long row: offsets, and sums of many stages."""
    g = draw(3, 50000, 1)
    check(muon.orthogonalize(g), g)
    g = draw(40001, 5, 2)
    check(muon.orthogonalize(g), g)
