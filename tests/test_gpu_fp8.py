"""Block-scaled e4m3 quantization and the linear layer's three products,
against the 64-bit statements in ``oracle.fp8``."""

import numpy as np
import pytest
import torch

from oracle import fp8 as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
# half a unit in the last place, relative; fp16's least subnormal, halved
ROUND = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
TINY = {"fp32": 2.0 ** -149, "bf16": 2.0 ** -134, "fp16": 2.0 ** -25}


@pytest.fixture(scope="module")
def fp8():
    from block_wise_dynamic_gb300 import build

    build.build()
    from block_wise_dynamic_gb300 import fp8 as m

    return m


def np64(t):
    return t.detach().double().cpu().numpy()


def draw(shape, seed, kind, std=1.0, loud=True):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal(shape) * std
    if loud and x.size:
        x *= np.exp(rng.standard_normal((shape[0], 1)))  # rows of different sizes
        x[:, rng.random(shape[1]) < 0.02] *= 30
    return torch.from_numpy(x).to(DEV).to(TYPES[kind])


def scale_bytes(scales, count, length):
    """The documented place of each line's and block's byte."""
    s = scales.cpu().numpy()
    groups = -(-(-(-length // 128)) // 4)
    r, k = np.meshgrid(np.arange(count), np.arange(-(-length // 128)), indexing="ij")
    return s[((r // 128) * groups + k // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + k % 4].astype(np.int64)


def check_quantized(q, x, blocks):
    """Codes and scales of every form that `blocks` has, exactly."""
    rows, cols = x.shape
    xs = np64(x)
    table = ref.e4m3_values()
    forms = {"rows": [("row", 1, 128)], "cols": [("col", 128, 1)], "both": [("row", 1, 128), ("col", 128, 1)],
             "tiles": [("row", 128, 128), ("col", 128, 128)]}[blocks]
    for name, br, bc in forms:
        want, e = ref.quantize(xs, br, bc)
        codes, scales = getattr(q, name + "_codes"), getattr(q, name + "_scales")
        by_line = np.repeat(np.repeat(e, br, 0), bc, 1)[:rows, :cols]
        got = scale_bytes(scales, rows, cols)[:, np.arange(cols) // 128] if name == "row" \
            else scale_bytes(scales, cols, rows)[:, np.arange(rows) // 128].T
        assert np.array_equal(got, np.where(by_line == 128, 255, by_line + 127))
        v = table[codes.cpu().numpy()[:, :cols]] * np.exp2(np.where(by_line == 128, 0, by_line).astype(np.float64))
        assert np.array_equal(v, want, equal_nan=True)
        back = q.dequantize("rows" if name == "row" else "cols", torch.float32)
        assert np.array_equal(np64(back), want.astype(np.float32).astype(np.float64), equal_nan=True)


@pytest.mark.parametrize("blocks", ["rows", "cols", "both", "tiles"])
@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("shape", [(1, 1), (1, 128), (3, 129), (128, 128), (129, 127), (200, 1000), (33, 516), (257, 2052)])
def test_quantize(fp8, shape, kind, blocks):
    x = draw(shape, 1, kind)
    check_quantized(fp8.quantize(x, blocks), x, blocks)


@pytest.mark.parametrize("blocks", ["rows", "cols", "both", "tiles"])
@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("cols", [1, 17, 63, 65, 100, 129, 300, 513, 1003])
def test_rows_are_padded_with_zeros(fp8, cols, kind, blocks):
    """A product reads whole rows: what lies past a matrix must not count."""
    x = draw((150, cols), cols, kind)
    size = fp8.quantize(x, blocks).buffer.numel()
    for _ in range(4):  # memory that held something else
        torch.full((size,), 0x7F, dtype=torch.uint8, device=DEV)
    q = fp8.quantize(x, blocks)
    for codes in (q.row_codes, q.col_codes):
        if codes is not None:
            assert codes.shape == (150, fp8._pitch(cols))
            assert not codes[:, cols:].any()


@pytest.mark.parametrize("blocks", ["both", "tiles"])
def test_quantize_special_values(fp8, blocks):
    x = torch.randn(300, 700, device=DEV)
    x[:128, :128] = 0.0
    x[5, 130] = float("nan")
    x[140, 300] = float("inf")
    x[141, 400] = -float("inf")
    x[128:256, 512:640] *= 2.0 ** -140           # subnormal maximum
    x[10, 512:640] = torch.finfo(torch.float32).max
    x[11, 384:512] = torch.tensor([448.0, 447.9, 17.0, 18.0, 19.0, 0.001, 2.0 ** -10, 3 * 2.0 ** -11] * 16)  # ties
    x[12, 384] = float(np.nextafter(np.float32(448), np.float32(1e9)))
    x[299, 640:] = -0.0
    check_quantized(fp8.quantize(x, blocks), x, blocks)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("offset,ld", [(0, 300), (1, 300), (4, 300), (8, 264), (2, 261)])
def test_quantize_strided(fp8, offset, ld, kind):
    base = draw((1, 150 * 320), 2, kind, loud=False).view(-1)
    x = torch.as_strided(base, (140, 257), (ld, 1), offset)
    check_quantized(fp8.quantize(x, "both"), x, "both")
    t = draw((257, 140), 3, kind).t()             # columns contiguous: copied by the call
    check_quantized(fp8.quantize(t, "both"), t, "both")


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("shape", [(1, 5), (128, 128), (1000, 261), (0, 7)])
def test_col_sums(fp8, shape, kind):
    x = draw(shape, 4, kind)
    q, s = fp8.quantize(x, "cols", col_sums=True)
    xs = np64(x)
    # fp32 sums of `rows` terms, then one rounding
    bound = shape[0] * 2.0 ** -24 * np.abs(xs).sum(0) + ROUND[kind] * np.abs(xs.sum(0)) + TINY[kind]
    assert np.all(np.abs(np64(s) - xs.sum(0)) <= bound)
    if shape[0]:
        check_quantized(q, x, "cols")


def near(got, want, size, k, kind):
    """Within the sums' and the result's rounding.  The matrix instruction adds
    32 products at a time into an fp32 sum and truncates: a unit of the last
    place of a running sum that never exceeds `size` for each addition.  For
    fp32 results there are 64 of them to a stretch of 2,048 products, and the
    stretches are added up to nearest; 16-bit results take all in one."""
    steps = 64 + -(-k // 2048) if kind == "fp32" else -(-k // 32) + 1
    bound = steps * 2.0 ** -23 * size + ROUND[kind] * np.abs(want) + TINY[kind]
    bad = np.abs(np64(got) - want) > bound
    assert not bad.any(), (np.argwhere(bad)[:4], np64(got)[bad][:4], want[bad][:4])
    norm = np.linalg.norm(want)
    assert np.linalg.norm(np64(got) - want) <= (1e-6 + 2 * ROUND[kind]) * norm + TINY[kind] * want.size


SIZES = [(1, 1, 1), (1, 128, 128), (2, 5, 300), (16, 256, 512), (17, 130, 1000), (64, 1024, 640), (100, 129, 2049), (128, 128, 128),
         (129, 257, 384), (300, 520, 1111), (513, 64, 4096), (70, 3000, 96), (260, 1000, 8300), (1000, 777, 130)]


@pytest.mark.parametrize("trans_a,trans_b", [(False, False), (False, True), (True, False), (True, True)])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_matmul_orders(fp8, m, n, k, trans_a, trans_b):
    a = draw((k, m) if trans_a else (m, k), 5, "bf16")
    b = draw((k, n) if trans_b else (n, k), 6, "bf16")
    aq, bq = fp8.quantize(a, "cols" if trans_a else "rows"), fp8.quantize(b, "cols" if trans_b else "rows")
    av, bv = ref.quantize(np64(a), *((128, 1) if trans_a else (1, 128)))[0], ref.quantize(np64(b), *((128, 1) if trans_b else (1, 128)))[0]
    av, bv = av.T if trans_a else av, bv.T if trans_b else bv
    for kind in ("fp32", "bf16"):
        got = fp8.matmul(aq, bq, trans_a, trans_b, dtype=TYPES[kind])
        near(got, av @ bv.T, np.abs(av) @ np.abs(bv).T, k, kind)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("trans_a,trans_b", [(False, False), (False, True), (True, False), (True, True)])
@pytest.mark.parametrize("m,n,k", [(4096, 4900, 200), (4000, 5001, 1300), (9000, 2300, 2100)])
def test_matmul_of_several_waves(fp8, m, n, k, trans_a, trans_b, kind):
    """More tiles than the device works on at a time, and a last wave of few."""
    a = draw((k, m) if trans_a else (m, k), 31, "bf16")
    b = draw((k, n) if trans_b else (n, k), 32, "bf16")
    aq, bq = fp8.quantize(a, "cols" if trans_a else "rows"), fp8.quantize(b, "cols" if trans_b else "rows")
    bias = draw((1, n), 33, kind, loud=False).view(-1)
    av, bv = (q.dequantize("cols" if t else "rows", torch.float32).double() for q, t in ((aq, trans_a), (bq, trans_b)))
    av, bv = av.t() if trans_a else av, bv.t() if trans_b else bv
    got = fp8.matmul(aq, bq, trans_a, trans_b, bias=bias, dtype=TYPES[kind])
    near(got, np64(av @ bv.t() + bias.double()), np64(av.abs() @ bv.abs().t() + bias.double().abs()), k, kind)


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_linear(fp8, m, n, k, bias, kind):
    x, w = draw((m, k), 7, kind), draw((n, k), 8, kind, 0.02, loud=False)
    b = draw((1, n), 9, kind, loud=False).view(-1) if bias else None
    got = fp8.linear(x, fp8.quantize(w, "tiles"), b)
    want, size = ref.linear(np64(x), np64(w), None if b is None else np64(b))
    near(got, want, size + (0 if b is None else np.abs(np64(b))), k, kind)


# few rows over a long summed axis: every part of a cluster goes round its
# stages several times
LONG = [(1, 200, 20000), (3, 11008, 4096), (16, 300, 33000), (2, 40000, 2300), (33, 129, 20000), (64, 2000, 9000), (128, 130, 30011)]


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("m,n,k", LONG)
def test_few_rows_long_sums(fp8, m, n, k, kind):
    x, w = draw((m, k), 21, kind), draw((n, k), 22, kind, 0.02, loud=False)
    got = fp8.linear(x, fp8.quantize(w, "tiles"))
    near(got, *ref.linear(np64(x), np64(w)), k, kind)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("m,n,k", [(300, 516, 260), (300, 518, 262), (300, 517, 261), (290, 514, 132), (70, 12, 20)])
def test_rows_of_other_alignments(fp8, m, n, k, kind):
    """Rows of 8, 4 and 2 bytes' alignment, read by the quantizers and written
    by the products, also from inside a larger matrix."""
    x, w, dy = draw((m, k), 24, kind), draw((n, k), 25, kind, 0.02, loud=False), draw((m, n), 26, kind, 0.01)
    for blocks in ("rows", "both", "tiles"):
        check_quantized(fp8.quantize(x, blocks), x, blocks)
        check_quantized(fp8.quantize(x[3:, 1:], blocks), x[3:, 1:], blocks)
        check_quantized(fp8.quantize(x[:, 2:k - 1], blocks), x[:, 2:k - 1], blocks)
    wq = fp8.quantize(w, "tiles")
    y, xq = fp8.forward(x, wq)
    dx, dw, _ = fp8.backward(dy, xq, wq)
    near(y, *ref.linear(np64(x), np64(w)), k, kind)
    (rx, rw, _), (sx, sw) = ref.linear_backward(np64(dy), np64(x), np64(w))
    near(dx, rx, sx, n, kind)
    near(dw, rw, sw, m, kind)


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_backward(fp8, m, n, k, kind):
    x, w, dy = draw((m, k), 10, kind), draw((n, k), 11, kind, 0.02, loud=False), draw((m, n), 12, kind, 0.01)
    wq = fp8.quantize(w, "tiles")
    y, xq = fp8.forward(x, wq)
    dx, dw, db = fp8.backward(dy, xq, wq, need_bias=True)
    near(y, *ref.linear(np64(x), np64(w)), k, kind)
    (rx, rw, rb), (sx, sw) = ref.linear_backward(np64(dy), np64(x), np64(w))
    near(dx, rx, sx, n, kind)
    near(dw, rw, sw, m, kind)
    dys = np64(dy)
    assert np.all(np.abs(np64(db) - rb) <= m * 2.0 ** -24 * np.abs(dys).sum(0) + ROUND[kind] * np.abs(rb) + TINY[kind])


def test_gradients_against_differences(fp8):
    """On small whole numbers quantization is exact, so differences of the
    layer's own forward pass are exact too."""
    g = torch.Generator(DEV).manual_seed(3)
    x, w, dy = (torch.randint(-4, 5, s, generator=g, device=DEV).float() for s in ((19, 150), (23, 150), (19, 23)))
    layer = fp8.Fp8Linear(150, 23, device=DEV, dtype=torch.float32)
    with torch.no_grad():
        layer.weight.copy_(w)
    xr = x.clone().requires_grad_()
    layer(xr).backward(dy)

    def loss():
        return float((layer(x).double() * dy.double()).sum())

    with torch.no_grad():
        base = loss()
        for r, c in ((0, 0), (7, 149), (18, 77)):
            x[r, c] += 2
            assert loss() - base == 2 * float(xr.grad[r, c])
            x[r, c] -= 2
        for r, c in ((0, 0), (22, 149), (11, 5)):
            layer.weight[r, c] += 2
            assert loss() - base == 2 * float(layer.weight.grad[r, c])
            layer.weight[r, c] -= 2
        for c in (0, 22):
            layer.bias[c] += 2
            assert loss() - base == 2 * float(layer.bias.grad[c])
            layer.bias[c] -= 2


def test_module_shapes_and_partial_gradients(fp8):
    layer = fp8.Fp8Linear(96, 40, device=DEV)
    x = torch.randn(2, 3, 96, device=DEV, dtype=torch.bfloat16)
    y = layer(x)
    assert y.shape == (2, 3, 40) and y.dtype == torch.bfloat16
    y.sum().backward()
    assert layer.weight.grad.shape == (40, 96) and torch.equal(layer.bias.grad, torch.full_like(layer.bias, 6.0))
    frozen = fp8.Fp8Linear(96, 40, bias=False, device=DEV)
    frozen.weight.requires_grad_(False)
    xr = x.clone().requires_grad_()
    frozen(xr).sum().backward()
    assert xr.grad.shape == x.shape and frozen.weight.grad is None


@pytest.mark.parametrize("m,n,k", [(0, 5, 7), (5, 0, 7), (5, 7, 0)])
def test_empty(fp8, m, n, k):
    x, w = torch.randn(m, k, device=DEV), torch.randn(n, k, device=DEV)
    bias = torch.randn(n, device=DEV)
    wq = fp8.quantize(w, "tiles")
    y, xq = fp8.forward(x, wq, bias)
    assert torch.equal(y, bias.expand(m, n) if k == 0 else torch.empty(m, n, device=DEV))
    dx, dw, db = fp8.backward(torch.ones(m, n, device=DEV), xq, wq, need_bias=True)
    assert torch.equal(dx, torch.zeros(m, k, device=DEV)) and torch.equal(dw, torch.zeros(n, k, device=DEV))
    assert torch.equal(db, torch.full((n,), float(m), device=DEV))


@pytest.mark.parametrize("m", [3, 40, 300])
def test_non_finite_reaches_what_it_should(fp8, m):
    """A NaN or infinity of x makes its own row of y NaN, one of w its tile's
    128 columns, and no other element."""
    x, w = draw((m, 400), 13, "bf16"), draw((300, 400), 14, "bf16", 0.02)
    clean = fp8.linear(x, fp8.quantize(w, "tiles"))
    x2, w2 = x.clone(), w.clone()
    x2[1, 399] = float("inf")
    y = fp8.linear(x2, fp8.quantize(w, "tiles"))
    assert torch.isnan(y[1]).all()
    keep = torch.arange(m, device=DEV) != 1
    assert torch.equal(y[keep], clean[keep])
    w2[140, 7] = float("nan")
    y = fp8.linear(x, fp8.quantize(w2, "tiles"))
    assert torch.isnan(y[:, 128:256]).all()
    assert torch.equal(y[:, :128], clean[:, :128]) and torch.equal(y[:, 256:], clean[:, 256:])


def test_same_result_every_time_and_on_another_stream(fp8):
    x, w = draw((700, 3000), 15, "bf16"), draw((900, 3000), 16, "bf16", 0.02)
    wq = fp8.quantize(w, "tiles")
    first = fp8.linear(x, wq)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for _ in range(5):
            again = fp8.linear(x, wq)
    s.synchronize()
    assert torch.equal(first, again)
    import block_wise_dynamic_gb300 as bwd

    bwd.check_device(0)


@pytest.mark.parametrize("handle", [False, True])
def test_stream_argument(fp8, handle):
    """A given stream is used for everything, copies of strided inputs and
    temporaries among it."""
    s = torch.cuda.Stream()
    x, w = draw((40, 300), 27, "bf16").t(), draw((500, 40), 28, "bf16", 0.02)
    want_w = fp8.quantize(w, "tiles")
    y, xq = fp8.forward(x, want_w)
    want = [y, *fp8.backward(y, xq, want_w, need_bias=True), fp8.linear(x, want_w), xq.dequantize("cols")]
    torch.cuda.synchronize()
    at = s.cuda_stream if handle else s
    for _ in range(3):
        wq = fp8.quantize(w, "tiles", stream=at)
        y, xq = fp8.forward(x, wq, stream=at)
        got = [y, *fp8.backward(y, xq, wq, need_bias=True, stream=at), fp8.linear(x, wq, stream=at), xq.dequantize("cols", stream=at)]
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_graph_capture(fp8):
    x, w = draw((48, 512), 17, "bf16"), draw((640, 512), 18, "bf16", 0.02)
    wq = fp8.quantize(w, "tiles")
    want = fp8.linear(x, wq)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        fp8.linear(x, wq)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = fp8.linear(x, wq)
    x.mul_(2.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want * 2)


def test_refusals(fp8):
    x = torch.randn(4, 8, device=DEV)
    w = fp8.quantize(torch.randn(6, 8, device=DEV), "tiles")
    with pytest.raises(ValueError):
        fp8.quantize(x, "columns")
    with pytest.raises(ValueError):
        fp8.quantize(x, "rows", col_sums=True)
    with pytest.raises(ValueError):
        fp8.quantize(x.cpu(), "rows")
    with pytest.raises(TypeError):
        fp8.quantize(x.double(), "rows")
    with pytest.raises(ValueError):
        fp8.linear(x[:, :7], w)
    with pytest.raises(TypeError):
        fp8.linear(x, torch.randn(6, 8, device=DEV))
    with pytest.raises(TypeError):
        fp8.linear(x, w, torch.zeros(6, device=DEV, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        fp8.linear(x, w, torch.zeros(5, device=DEV))
    with pytest.raises(ValueError):
        fp8.linear(x, fp8.quantize(torch.randn(6, 8, device=DEV), "cols"))  # blocks along the wrong axis
    with pytest.raises(ValueError):
        fp8.matmul(fp8.quantize(x, "rows"), fp8.quantize(torch.randn(6, 9, device=DEV), "rows"))
    xq = fp8.quantize(x, "rows")
    with pytest.raises(ValueError):
        fp8.backward(torch.ones(4, 6, device=DEV), xq, w)
    with pytest.raises(ValueError):
        fp8.backward(torch.ones(4, 5, device=DEV), xq, w)


def test_offsets_past_2_to_31(fp8):
    """A matrix of more than 2^31 elements, checked in its last rows."""
    rows, cols = (1 << 18) + 40, 8256
    free, _ = torch.cuda.mem_get_info()
    if free < 24 << 30:
        pytest.skip("needs 24 GB")
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    tail = draw((40, cols), 19, "bf16")
    x[-40:] = tail
    w = draw((24, cols), 20, "bf16", 0.02)
    got = fp8.linear(x, fp8.quantize(w, "tiles"))
    want, size = ref.linear(np64(tail), np64(w))
    near(got[-40:], want, size, cols, "bf16")
    assert not got[:-40].any()
    dw = fp8.matmul(fp8.quantize(got, "cols"), fp8.quantize(x, "cols"), True, True)
    # the last 40 rows are the whole of the last block of 128 rows (2^18 is a multiple of 128)
    gv = ref.quantize(np64(got[-40:]), 128, 1)[0]
    xv = ref.quantize(np64(tail), 128, 1)[0]
    near(dw, gv.T @ xv, np.abs(gv).T @ np.abs(xv), rows, "bf16")


@pytest.mark.parametrize("m", [1, 16, 40, 64, 300])
def test_calls_in_a_row_see_each_others_results(fp8, m):
    """Kernels may begin before the one ahead has ended: what one call writes
    and the next reads, with nothing waited for in between."""
    n, k = 1024, 4096
    g = torch.Generator(DEV).manual_seed(23)
    ws = [torch.randn(n, k, generator=g, device=DEV).to(torch.bfloat16) for _ in range(8)]
    xs = [torch.randn(m, k, generator=g, device=DEV).to(torch.bfloat16) for _ in range(8)]
    want = []
    for w, x in zip(ws, xs):
        y, xq = fp8.forward(x, fp8.quantize(w, "tiles"))
        torch.cuda.synchronize()
        dx, dw, db = fp8.backward(y, xq, fp8.quantize(w, "tiles"), need_bias=True)
        torch.cuda.synchronize()
        want.append((y, dx, dw, db, fp8.linear(x, fp8.quantize(w, "rows"))))
        torch.cuda.synchronize()
    w, x = torch.empty_like(ws[0]), torch.empty_like(xs[0])
    got = []
    for i in range(8):
        w.copy_(ws[i])
        x.copy_(xs[i])
        wq = fp8.quantize(w, "tiles")
        y, xq = fp8.forward(x, wq)
        dx, dw, db = fp8.backward(y, xq, wq, need_bias=True)
        w.mul_(1.0)
        got.append((y, dx, dw, db, fp8.linear(x, fp8.quantize(w, "rows"))))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("trans_a,trans_b", [(False, False), (False, True), (True, False), (True, True)])
@pytest.mark.parametrize("m,n,k", [(65, 1, 4000), (128, 129, 4097), (353, 135, 9883), (130, 2049, 5000), (500, 1000, 8192), (1300, 70, 6143),
                                   (640, 900, 11000), (50, 1000, 9000)])
def test_few_tiles_and_long_sums(fp8, m, n, k, trans_a, trans_b, kind):
    """The summed axis in as many parts as there is room for."""
    a = draw((k, m) if trans_a else (m, k), 41, "bf16")
    b = draw((k, n) if trans_b else (n, k), 42, "bf16")
    aq, bq = fp8.quantize(a, "cols" if trans_a else "rows"), fp8.quantize(b, "cols" if trans_b else "rows")
    bias = draw((1, n), 43, kind, loud=False).view(-1)
    av, bv = (q.dequantize("cols" if t else "rows", torch.float32).double() for q, t in ((aq, trans_a), (bq, trans_b)))
    av, bv = av.t() if trans_a else av, bv.t() if trans_b else bv
    got = fp8.matmul(aq, bq, trans_a, trans_b, bias=bias, dtype=TYPES[kind])
    near(got, np64(av @ bv.t() + bias.double()), np64(av.abs() @ bv.abs().t() + bias.double().abs()), k, kind)
    assert torch.equal(got, fp8.matmul(aq, bq, trans_a, trans_b, bias=bias, dtype=TYPES[kind]))


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("m,n,k", [(700, 600, 500), (2048, 1024, 1024), (4096, 1024, 640), (333, 3000, 1111), (5000, 2200, 2100), (300, 2176, 300)])
def test_backward_of_two_products_in_one_launch(fp8, m, n, k, kind):
    """The two products' tiles follow one another: each on its own, bit for
    bit, whatever its neighbour's sizes and row alignment."""
    x, w, dy = draw((m, k), 51, kind), draw((n, k), 52, kind, 0.02, loud=False), draw((m, n), 53, kind, 1e-3)
    wq = fp8.quantize(w, "tiles")
    xq, dyq = fp8.quantize(x, "cols"), fp8.quantize(dy, "both")
    dx, dw, db = fp8.backward(dy, xq, wq, need_bias=True)
    assert torch.equal(dx, fp8.matmul(dyq, wq, trans_b=True))
    assert torch.equal(dw, fp8.matmul(dyq, xq, True, True))
    assert torch.equal(db, fp8.quantize(dy, "cols", col_sums=True)[1])
    wv, xv = wq.dequantize("cols", torch.float32).double(), xq.dequantize("cols", torch.float32).double()
    rows, cols = dyq.dequantize("rows", torch.float32).double(), dyq.dequantize("cols", torch.float32).double()
    near(dx, np64(rows @ wv), np64(rows.abs() @ wv.abs()), n, kind)
    near(dw, np64(cols.t() @ xv), np64(cols.abs().t() @ xv.abs()), m, kind)
