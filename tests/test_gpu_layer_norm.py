"""Layer norm forward and backward against the 64-bit statement."""

import numpy as np
import pytest
import torch

from oracle import layer_norm as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
U = 2.0 ** -24
# half a step relative to the value, and half the least subnormal
ROUND = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
TINY = {"fp32": 2.0 ** -149, "bf16": 2.0 ** -134, "fp16": 2.0 ** -25}


@pytest.fixture(scope="module")
def norm():
    from block_wise_dynamic_gb300 import build

    build.build()
    from block_wise_dynamic_gb300 import norm as m

    return m


def np64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def name_of(dtype):
    return next(k for k, v in TYPES.items() if v == dtype)


def draw(rows, width, seed, kind, offset=True):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, width)) * np.exp(rng.standard_normal((rows, 1)))
    if offset:
        x += 3.0 * rng.standard_normal((rows, 1))
    return torch.from_numpy(x).to(DEV).to(TYPES[kind])


def rounded(want, error, dtype):
    """How far a result may be from `want`, when it is off by `error` before it is rounded."""
    kind = name_of(dtype)
    return error + ROUND[kind] * (np.abs(want) + error) + TINY[kind]


def near(got, want, bound):
    got = np64(got)
    assert got.shape == want.shape and np.isfinite(got).all()
    over = np.abs(got - want) - bound
    assert over.max(initial=-1.0) <= 0, f"{over.max()} beyond the bound at {np.unravel_index(over.argmax(), over.shape)}"


def check_forward(x, gamma, beta, y, mean, rstd, eps):
    """A row's sum has chains of 16 additions in a thread and of 10 between
    threads; with the division and slack, the mean is within 40 U of the mean
    magnitude, and so on."""
    xs, g, b = np64(x).reshape(-1, x.shape[-1]), np64(gamma), np64(beta)
    want, m, r = ref.forward(xs, g, b, eps)
    off_mean = 40 * U * np.abs(xs).mean(1)
    # variance: of values centred by a mean off by off_mean, summed and divided; half of it in rstd, which takes two more roundings
    off_rstd = 0.5 * (60 * U + off_mean ** 2 * r ** 2 + 2 * off_mean * r * 4 * U) + 4 * U
    xh = (xs - m[:, None]) * r[:, None]
    off = (off_mean * r)[:, None] * (1 + 4 * U) + np.abs(xh) * (off_rstd + 4 * U)[:, None]
    if g is not None:
        off = off * np.abs(g)
    off = off + 2 * U * (np.abs(want) + off)
    near(y.reshape(want.shape), want, rounded(want, off, y.dtype))
    if mean is not None:
        near(mean, m, off_mean + U * np.abs(m))
        near(rstd, r, r * (off_rstd + U))


def check_backward(dy, x, gamma, mean, rstd, dx, dgamma, dbeta):
    """For the statistics as they were handed in."""
    xs, ds, g = np64(x).reshape(-1, x.shape[-1]), np64(dy).reshape(-1, x.shape[-1]), np64(gamma)
    m, r = np64(mean), np64(rstd)
    want_x, want_g, want_b = ref.backward(ds, xs, g, m, r)
    xh = np.abs((xs - m[:, None]) * r[:, None])
    h = np.abs(ds if g is None else ds * g)
    if dx is not None:
        mean_h, mean_hx = h.mean(1, keepdims=True), (h * xh).mean(1, keepdims=True)
        off = r[:, None] * U * (6 * h + 46 * mean_h + 52 * xh * mean_hx)
        near(dx.reshape(want_x.shape), want_x, rounded(want_x, off, dx.dtype))
    # a column's sum: rows of one CTA, its warps, every eighth of the CTAs' parts, eight of those
    chain = len(xs) / 152 + 1 + 8 + 160 * 4 / 8 + 8
    for got, want, size in ((dgamma, want_g, (np.abs(ds) * xh).sum(0)), (dbeta, want_b, np.abs(ds).sum(0))):
        if got is not None:
            near(got, want, rounded(want, U * (chain + 4) * size, got.dtype))


SIZES = [(1, 1), (1, 4096), (3, 7), (5, 33), (1, 16384), (300, 64), (77, 512), (77, 513), (129, 1003), (40, 1024), (33, 4096), (9, 8192),
         (9, 8200), (5, 11008), (3, 16383), (2000, 130), (4000, 1000), (2500, 1003), (3000, 520), (700, 4100), (700, 4096), (900, 8193),
         (700, 9001), (700, 6144), (700, 12288), (650, 16384), (640, 13001)]


@pytest.mark.parametrize("kind,vectors", [("fp32", "fp32"), ("bf16", "fp32"), ("bf16", "bf16"), ("fp16", "fp32"), ("fp16", "fp16")])
@pytest.mark.parametrize("rows,width", SIZES)
def test_both_passes(norm, rows, width, kind, vectors):
    x, dy = draw(rows, width, 1, kind), draw(rows, width, 2, kind, offset=False)
    gamma = draw(1, width, 3, vectors, offset=False)[0] + 1
    beta = draw(1, width, 4, vectors, offset=False)[0]
    y, mean, rstd = norm.forward(x, gamma, beta, 1e-5)
    assert y.dtype == x.dtype and mean.shape == rstd.shape == (rows,)
    check_forward(x, gamma, beta, y, mean, rstd, 1e-5)
    dx, dgamma, dbeta = norm.backward(dy, x, gamma, mean, rstd)
    assert dx.dtype == x.dtype and dgamma.dtype == dbeta.dtype == gamma.dtype
    check_backward(dy, x, gamma, mean, rstd, dx, dgamma, dbeta)
    again = norm.backward(dy, x, gamma, mean, rstd)
    assert all(torch.equal(a, b) for a, b in zip(again, (dx, dgamma, dbeta)))


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("off,pitch", [(0, 8), (1, 0), (1, 3), (2, 2), (4, 4), (0, 1), (7, 9)])
@pytest.mark.parametrize("rows,width", [(37, 96), (37, 1024), (37, 9000), (2000, 1001), (700, 4098), (650, 9003)])
def test_strides_and_alignment(norm, rows, width, off, pitch, kind):
    """Rows with a pitch, and starts off every boundary; what lies between is left alone."""
    flat = torch.full((off + rows * (width + pitch),), 1e4, dtype=TYPES[kind], device=DEV)
    x = flat[off:off + rows * (width + pitch)].view(rows, width + pitch)[:, :width]
    x.copy_(draw(rows, width, 5, kind))
    dy_flat = torch.zeros_like(flat)
    dy = dy_flat[off:off + rows * (width + pitch)].view(rows, width + pitch)[:, :width]
    dy.copy_(draw(rows, width, 6, kind))
    before = flat.clone()
    gamma = draw(1, width + 1, 7, "fp32")[0][1:]
    y, mean, rstd = norm.forward(x, gamma, None)
    check_forward(x, gamma, None, y, mean, rstd, norm.EPS)
    grads = norm.backward(dy, x, gamma, mean, rstd)
    check_backward(dy, x, gamma, mean, rstd, *grads)
    assert torch.equal(flat, before)
    # a view whose columns are not contiguous is copied
    t = draw(width, rows, 8, kind).t()
    check_forward(t, gamma, None, *norm.forward(t, gamma, None), norm.EPS)


def test_what_is_not_needed(norm):
    x, dy = draw(50, 300, 1, "bf16"), draw(50, 300, 2, "bf16")
    y, mean, rstd = norm.forward(x)
    assert norm.forward(x, need_stats=False)[1:] == (None, None)
    check_forward(x, None, None, y, mean, rstd, norm.EPS)
    full = norm.backward(dy, x, None, mean, rstd, vector_dtype=torch.bfloat16)
    check_backward(dy, x, None, mean, rstd, *full)
    assert full[1].dtype == torch.bfloat16
    for needs in [(True, False, False), (False, True, False), (False, False, True), (False, True, True), (False, False, False)]:
        got = norm.backward(dy, x, None, mean, rstd, *needs, vector_dtype=torch.bfloat16)
        for g, f, need in zip(got, full, needs):
            assert (g is None) if not need else torch.equal(g, f)


def test_leading_dimensions_and_nothing(norm):
    x = draw(6, 40, 1, "fp32").view(2, 3, 40)
    gamma = torch.ones(40, device=DEV)
    y, mean, rstd = norm.forward(x, gamma)
    assert y.shape == x.shape and mean.shape == (6,)
    assert norm.backward(x, x, gamma, mean, rstd)[0].shape == x.shape
    none = torch.empty(0, 40, device=DEV)
    y, mean, rstd = norm.forward(none, gamma)
    dx, dgamma, dbeta = norm.backward(none, none, gamma, mean, rstd)
    assert y.shape == dx.shape == (0, 40) and not dgamma.any() and not dbeta.any()


def test_special_rows(norm):
    """Constant rows, rows with an infinity or a NaN, offsets a million times the spread, huge and tiny rows."""
    x = draw(8, 700, 1, "fp32", offset=False)
    x[1] = 3.25
    x[2, 5] = float("inf")
    x[3, 699] = float("nan")
    x[4] += 1e4
    x[5] *= 1e15
    x[6] *= 1e-25
    x[7] = 0.0
    beta = torch.linspace(-1, 1, 700, device=DEV)
    y, mean, rstd = norm.forward(x, None, beta)
    assert torch.equal(y[1], beta) and torch.equal(y[7], beta) and y[2].isnan().any() and y[3].isnan().all()
    keep = [0, 1, 4, 5, 6, 7]
    check_forward(x[keep], None, beta, y[keep], mean[keep], rstd[keep], norm.EPS)


def test_many_rows(norm):
    """More elements than 2^31, and rows beyond the grid."""
    if torch.cuda.get_device_properties(0).total_memory < 60 << 30:
        pytest.skip("needs 40 GB")
    rows, width = (1 << 31) // 1000 + 10, 1000
    x = torch.empty((rows, width), dtype=torch.bfloat16, device=DEV).normal_(generator=torch.Generator(DEV).manual_seed(0))
    y, mean, rstd = norm.forward(x)
    dx = norm.backward(x, x, None, mean, rstd, need_gamma=False, need_beta=False)[0]
    for part in (slice(0, 50), slice(rows - 50, rows)):
        check_forward(x[part], None, None, y[part], mean[part], rstd[part], norm.EPS)
        check_backward(x[part], x[part], None, mean[part], rstd[part], dx[part], None, None)


def test_module(norm):
    m = norm.LayerNorm(130).to(DEV)
    with torch.no_grad():
        m.weight.uniform_(0.5, 1.5)
        m.bias.uniform_(-1, 1)
    x = draw(20, 130, 1, "bf16").view(4, 5, 130).requires_grad_()
    y = m(x)
    dy = draw(20, 130, 2, "bf16").view(4, 5, 130)
    y.backward(dy)
    _, mean, rstd = norm.forward(x, m.weight, m.bias)
    check_backward(dy, x, m.weight, mean, rstd, x.grad, m.weight.grad, m.bias.grad)
    with torch.no_grad():
        assert torch.equal(m(x), y)
    # a gradient that is one value everywhere has no strides
    x.grad = None
    m(x).sum().backward()
    assert x.grad.shape == x.shape
    x2 = x.detach().requires_grad_()
    (g,) = torch.autograd.grad(m(x2).sum(), x2, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivatives"):
        g.sum().backward()
    plain = norm.LayerNorm(16, bias=False, dtype=torch.bfloat16)
    x3 = torch.ones(2, 16, dtype=torch.bfloat16, device=DEV)
    plain(x3).sum().backward()
    assert plain.bias is None and plain.weight.grad.dtype == torch.bfloat16


def test_gradient_is_the_differences(norm):
    x, dy = draw(3, 9, 1, "fp32"), draw(3, 9, 2, "fp32")
    gamma, beta = draw(1, 9, 3, "fp32")[0], draw(1, 9, 4, "fp32")[0]
    _, mean, rstd = norm.forward(x, gamma, beta)
    dx = np64(norm.backward(dy, x, gamma, mean, rstd)[0])
    xs, ds = np64(x), np64(dy)
    for at in np.ndindex(xs.shape):
        sides = []
        for h in (1e-6, -1e-6):
            moved = xs.copy()
            moved[at] += h
            sides.append((ref.forward(moved, np64(gamma), np64(beta))[0] * ds).sum())
        # the statistics are rounded to fp32: a few parts in 10^6 of what enters a row's gradient
        size = np64(rstd)[at[0]] * np.abs(ds[at[0]] * np64(gamma)).max() * 10
        assert abs((sides[0] - sides[1]) / 2e-6 - dx[at]) < 3e-6 * size


def test_streams_and_graphs(norm):
    x, dy = draw(64, 256, 1, "bf16"), draw(64, 256, 2, "bf16")
    gamma = torch.ones(256, device=DEV)
    want = norm.forward(x, gamma)
    want = want + norm.backward(dy, x, gamma, *want[1:])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y, mean, rstd = norm.forward(x, gamma, stream=side)
    grads = norm.backward(dy, x, gamma, mean, rstd, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((y, mean, rstd) + grads, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = norm.forward(x, gamma)
        out = out + norm.backward(dy, x, gamma, *out[1:])
    x.copy_(draw(64, 256, 3, "bf16"))
    graph.replay()
    torch.cuda.synchronize()
    check_forward(x, gamma, None, *out[:3], norm.EPS)
    check_backward(dy, x, gamma, out[1], out[2], *out[3:])


def test_two_streams_at_once(norm):
    x = [draw(rows, width, i, "bf16") for i, (rows, width) in enumerate(((900, 4096), (900, 1003), (40, 300)))]
    want = [norm.forward(a) for a in x]
    want = [w + norm.backward(a, a, None, *w[1:]) for a, w in zip(x, want)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in x]
    for _ in range(10):
        got = [norm.forward(a, stream=s) for a, s in zip(x, streams)]
        got = [g + norm.backward(a, a, None, *g[1:], stream=s) for a, g, s in zip(x, got, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))
