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


def squares_bound(g, steps, squares):
    """As error_bound, for a result whose last `squares` steps stay among m x m matrices (m rows of the wide form).

    P = a I + B, Q = P Q, A' = P A P, all of them polynomials of A.  An operand
    is off by d of its value; sums of 128 products leave the accumulator and
    are added up in fp32, so that a product is off by e = 2.02 d + 128 2e-10 +
    2^-24 (n / 128 + 4) of the sum of its terms' magnitudes.  With Frobenius
    norms F = |X|, |A| and |B| <= 4.8 |A|, and spectral norms of at most 1.47 of
    A, 3.45 of P and 1.5 of P A, what one step adds:
      the first A    e F^2 + d |A|
      B              t = 2.04 e |A|^2 + d |B|, and on the first P's diagonal 3.45 d
      P A            e |B| |A| + 1.5 d |A|, times |P|
      P (P A)        1.5 e |B| |A| + d |A'|
      both times B   3 t, and 3 3.45 d |A| for the first
    these last three times 2^1/2, as one half is the other's mirror image.  An
    error of A grows by 11.9 a step, the largest slope of s (a + b s + c s^2)^2.
    What moves X: P_k's error, 4.8 times A_k's and t, times |X_k| <= 1.21; Q's
    rounding and product, (d |Q| + e 3.45^k |B|) times X's spectral norm with
    |Q| <= 3.45^(k+1) m^1/2; each raised by 3.45 a step that follows; and Q X,
    e |Q| F.  X's own error before them is stretched by 4.3 a step.  Stored
    values (times 2^14, Q's divided by 4^k) are off by 2^-39 besides.  All to
    first order: a twentieth on top."""
    xs = ref.iterates(np64(g), steps)
    m, n = xs[0].shape
    start, least = steps - squares, 2.0 ** -39
    d = 2.0 ** -22 + 2.0 ** -30
    e = 2.02 * d + 2e-10 * 128 + 2.0 ** -24 * (n / 128 + 4)
    total = 2.0 ** -20 * np.linalg.norm(xs[0]) + least * (m * n) ** 0.5
    for x in xs[:start]:
        f = np.linalg.norm(x)
        total = 4.3 * total + 27 * e * f * f + 29 * d * f + 17.5 * least * (m * n) ** 0.5
    total *= 4.3 ** squares
    x0, f = np.linalg.norm(xs[start], 2), np.linalg.norm(xs[start])
    grams = [np.linalg.norm(x @ x.T) for x in xs[start:]]
    off = e * f * f + d * grams[0] + least * m
    for k in range(squares):
        a, b, first = grams[k], 4.8 * grams[k], 3.45 * d * (k == 0)
        t = 2.04 * e * a * a + d * b + least * m
        here = 1.21 * (4.8 * off + t + first * m ** 0.5)
        here += x0 * (3.45 ** (k + 1) * d * m ** 0.5 + 3.45 ** k * e * b + 4 ** k * least * m)
        total += 3.45 ** (squares - 1 - k) * here
        step = 3.45 * (e * b * a + 1.5 * d * a) + 1.5 * e * b * a + d * grams[k + 1] + 3 * (t + first * a) + 5 * least * m
        off = 11.9 * off + 2 ** 0.5 * step
    return 1.05 * (total + e * 3.45 ** squares * m ** 0.5 * f)


def check_wide(out, g, steps=5):
    """g: so many columns (or rows) that the last five steps (bf16) or three stay among the squares."""
    want = ref.orthogonalize(np64(g), steps)
    off = np.linalg.norm(np64(out) - want)
    bound = squares_bound(g, steps, min(steps, 5 if g.dtype == torch.bfloat16 else 3))
    bound += ROUND[g.dtype] * (np.linalg.norm(want) + bound) + TINY[g.dtype] * want.size ** 0.5
    assert out.shape == g.shape and out.dtype == g.dtype and off <= bound, (off, bound)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", [(1000, 2100), (2303, 1001), (130, 30000)])
def test_wide(muon, shape, dtype):
    for kind in ("gauss", "strong"):
        g = draw(*shape, 21, kind, TYPES[dtype])
        before = g.clone()
        out = muon.orthogonalize(g)
        check_wide(out, g)
        assert torch.equal(g, before)
        # what the two forms of the steps are said to leave, whatever the spectrum
        want = ref.orthogonalize(np64(g))
        most = {"fp32": 1e-4, "bf16": 2.0 ** -8 + 1e-3, "fp16": 2.0 ** -11 + 1e-4}[dtype]
        assert np.linalg.norm(np64(out) - want) < most * np.linalg.norm(want)


def test_a_little_wide(muon):
    """bf16 results take the squares from 1.25 columns to a row on."""
    check_wide(muon.orthogonalize(g := draw(1320, 1650, 22, "strong", torch.bfloat16)), g)
    check(muon.orthogonalize(g := draw(1320, 1649, 22, "strong", torch.bfloat16)), g)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6, 9])
def test_wide_batches(muon, steps, dtype):
    g = torch.stack([draw(300, 700, 30 + i, "strong" if i % 2 else "gauss", TYPES[dtype]) for i in range(9)])
    out = muon.orthogonalize(g, steps)
    for i in (0, 1, 8):
        check_wide(out[i], g[i], steps)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_special_wide_matrices(muon, dtype):
    kind = TYPES[dtype]
    g = torch.stack([draw(300, 700, 40 + i) for i in range(9)])
    g[4] *= {"fp32": 1e30, "bf16": 1e37, "fp16": 1e6}[dtype]
    g[5] *= {"fp32": 1e-20, "bf16": 1e-1, "fp16": 1e-1}[dtype]
    g = g.to(kind)
    want = muon.orthogonalize(g)
    g[1] = 0
    g[2, 3, 4] = float("nan")
    g[3, 0, 0] = float("inf")
    out = muon.orthogonalize(g)
    for i in (0, 4, 5, 6, 7, 8):
        assert torch.equal(out[i], want[i])
    assert not out[1].any() and out[2].isnan().all() and out[3].isnan().all()
    for i in (4, 5):
        check_wide(out[i], g[i])


@pytest.mark.parametrize("p_type,g_type", [("fp32", "fp32"), ("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16")])
def test_wide_step(muon, p_type, g_type):
    """Without momentum and from zeros a step leaves -lr rms n^1/2 times the orthogonalised gradient."""
    gs = [draw(*((300, 700) if i % 2 else (700, 300)), 50 + i, "strong", TYPES[g_type]) for i in range(10)]
    ps = [torch.zeros(g.shape, dtype=TYPES[p_type], device=DEV) for g in gs]
    ms = [torch.zeros(g.shape, device=DEV) for g in gs]
    args = muon.MuonArgs(ps, gs, ms)
    args.step(lr=0.5, momentum=0.0, nesterov=False, weight_decay=0.0, rms=0.25)
    factor = 0.125 * 700 ** 0.5
    for p, g, m in zip(ps, gs, ms):
        assert torch.equal(m, g.float())
        want = ref.orthogonalize(np64(g))
        off = np.linalg.norm(np64(p) / -factor - want)
        bound = squares_bound(g, 5, 5 if p_type == "bf16" else 3)
        bound += (ROUND[TYPES[p_type]] + 4 * U) * (np.linalg.norm(want) + bound) + TINY[TYPES[p_type]] / factor * want.size ** 0.5
        assert off <= bound, (off, bound)


def test_a_wide_graph_replays(muon):
    """The planes' factors and Q's diagonal are formed anew by each replay."""
    for dtype in (torch.bfloat16, torch.float32):
        g = draw(1001, 2303, 60, "strong", dtype)
        muon.orthogonalize(g)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = muon.orthogonalize(g)
        for seed, factor in ((61, 1.0), (62, 1e-3), (63, 40.0)):
            g.copy_((draw(1001, 2303, seed, "strong") * factor).to(dtype))
            graph.replay()
            assert torch.equal(out, muon.orthogonalize(g))


def test_parameters_that_move(muon):
    """A parameter whose storage is replaced between steps is updated where it lies then."""
    g = draw(64, 100, 70)
    a, b = (torch.nn.Parameter(draw(64, 100, 71)) for _ in range(2))
    one, two = muon.Muon([a], lr=0.1), muon.Muon([b], lr=0.1)
    for step in range(3):
        a.grad, b.grad = g * (step + 1), g * (step + 1)
        one.step()
        two.step()
        old = a.data
        kept = old.clone()
        a.data = old.clone()
        a.grad = b.grad = g
        one.step()
        two.step()
        assert torch.equal(old, kept) and torch.equal(a, b)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_whatever_the_workspace_held(muon, dtype):
    """Sides that end 1 to 64 short of a stage of 64, with every bit of the workspace set before (NaNs in all of its types)."""
    for count, shape in ((1, (910, 993)), (3, (1050, 1060)), (8, (290, 700)), (1, (961, 2500)), (2, (520, 1300)), (3, (40, 70)), (2, (289, 300))):
        gs = [draw(*shape, 80 + i, "strong", TYPES[dtype]) for i in range(count)]
        want = muon.orthogonalize(torch.stack(gs))
        ps = [torch.zeros(shape, dtype=TYPES[dtype], device=DEV) for _ in gs]
        ms = [torch.zeros(shape, device=DEV) for _ in gs]
        args = muon.MuonArgs(ps, gs, ms)
        args.work.fill_(255)
        args.step(lr=1.0, momentum=0.0, nesterov=False, rms=0.125)
        factor = 0.125 * max(shape) ** 0.5
        for p, o in zip(ps, want):
            assert p.isfinite().all()
            # two roundings and two ways to the same result
            off = np.linalg.norm(np64(p) / -factor - np64(o))
            assert off <= (2 * ROUND[TYPES[dtype]] + 1e-3 * (dtype == "bf16") + 2e-4) * np.linalg.norm(np64(o))
