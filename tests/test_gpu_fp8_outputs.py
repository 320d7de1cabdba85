"""The products' results inside larger memory, ``ldo`` elements between rows:
bit for bit those of a contiguous result, and nothing beside them is written."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
MARK = 0xA5


@pytest.fixture(scope="module")
def fp8():
    from block_wise_dynamic_gb300 import build

    build.build()
    from block_wise_dynamic_gb300 import fp8 as m

    return m


class Place:
    """A rows x cols matrix whose address and rows are `align` bytes past a
    multiple of 16, in the middle of marked memory."""

    def __init__(self, rows, cols, dtype, align, gap):
        e = dtype.itemsize
        self.rows, self.cols, self.dtype = rows, cols, dtype
        pitch = ((cols + gap) * e + 15) // 16 * 16 + align
        self.ld, start = pitch // e, 4096 + align
        self.whole = torch.full((start + rows * pitch + 4096,), MARK, dtype=torch.uint8, device=DEV)
        self.at = np.full(self.whole.numel(), True)  # bytes that no result may change
        for r in range(rows):
            self.at[start + r * pitch:start + r * pitch + cols * e] = False
        self.ptr = self.whole.data_ptr() + start
        self.view = self.whole[start:start + rows * pitch].view(rows, pitch)[:, :cols * e].contiguous

    def check(self, want, what):
        got = self.view().view(self.dtype)
        assert torch.equal(got, want), what
        beside = self.whole.cpu().numpy()[self.at]
        assert (beside == MARK).all(), what


def aligns(kind):
    return (0, 8, 4) if kind == "fp32" else (0, 8, 4, 2)


def draw(shape, seed, kind):
    g = torch.Generator(DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(TYPES[kind])


# up to 16 rows; few rows; a sum in parts; pairs with 128 and with 256 columns, with long sums and short ones, and a last
# wave of half tiles; a product over nothing
PRODUCTS = [(5, 300, 260), (16, 129, 1000), (40, 300, 520), (130, 200, 5000), (300, 520, 384), (33, 65, 4096), (4000, 2500, 256),
            (4000, 2501, 2100), (4900, 2300, 200), (70, 30, 0)]


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_matmul(fp8, m, n, k, kind):
    a, b, bias = draw((m, k), 1, "bf16"), draw((n, k), 2, "bf16"), draw((n,), 3, kind)
    aq, bq = fp8.quantize(a, "rows"), fp8.quantize(b, "rows")
    want = fp8.matmul(aq, bq, bias=bias, dtype=TYPES[kind])
    for align in aligns(kind):
        for gap in (0, 9):
            out = Place(m, n, TYPES[kind], align, gap)
            fp8._launch("bwd_fp8_matmul", a.device, None, m, n, k, aq._pointers[0], 0, aq._pointers[1], bq._pointers[0], 0,
                        bq._pointers[1], bias.data_ptr(), out.ptr, out.ld, fp8._GDT[TYPES[kind]])
            out.check(want, (align, gap))


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_linear(fp8, m, n, k, kind):
    x, w, bias = draw((m, k), 4, kind), draw((n, k), 5, kind), draw((n,), 6, kind)
    wq = fp8.quantize(w, "tiles")
    want = fp8.linear(x, wq, bias)
    work = torch.empty(max(1, fp8._forward_work(m, k)), dtype=torch.uint8, device=DEV)
    for align in aligns(kind):
        out = Place(m, n, TYPES[kind], align, 3)
        fp8._launch("bwd_fp8_linear", x.device, None, x.data_ptr(), fp8._GDT[TYPES[kind]], m, k, k, *wq._pointers[:2], n,
                    bias.data_ptr(), out.ptr, out.ld, None, None, work.data_ptr())
        out.check(want, align)


# both products in one launch, in two, and one of them over few tiles
@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("m,n,k", [(700, 600, 500), (5, 300, 260), (300, 70, 4096), (4100, 1024, 640), (5000, 2201, 2100)])
def test_backward(fp8, m, n, k, kind):
    x, w, dy = draw((m, k), 7, kind), draw((n, k), 8, kind), draw((m, n), 9, kind)
    wq, xq = fp8.quantize(w, "tiles"), fp8.quantize(x, "cols")
    dx, dw, db = fp8.backward(dy, xq, wq, need_bias=True)
    work = torch.empty(fp8._backward_work(m, n), dtype=torch.uint8, device=DEV)
    places = aligns(kind)
    for i, align in enumerate(places):
        at_x, at_w = Place(m, k, TYPES[kind], align, 3), Place(n, k, TYPES[kind], places[i - 1], 5)
        at_b = Place(1, n, TYPES[kind], align, 0)
        fp8._launch("bwd_fp8_linear_backward", x.device, None, dy.data_ptr(), fp8._GDT[TYPES[kind]], m, n, n, *wq._pointers[2:],
                    *xq._pointers[2:], k, at_x.ptr, at_x.ld, at_w.ptr, at_w.ld, at_b.ptr, work.data_ptr())
        at_x.check(dx, ("dx", align))
        at_w.check(dw, ("dw", align))
        at_b.check(db.view(1, n), ("db", align))
