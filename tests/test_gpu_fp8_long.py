"""fp32 results of few rows over sums so long that an accumulator would have to
take more than 2,048 products."""

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


@pytest.mark.parametrize("m,n,k", [(16, 20000, 131072), (1, 20000, 40000), (3, 300, 262144 + 77), (16, 129, 500000)])
def test_few_rows(fp8, m, n, k):
    """Positive terms, so that truncation only takes away.  The matrix
    instruction loses 1.9e-10 of a sum for each of its products: 3.8e-7 over a
    stretch of 2,048, and then the stretches' and the parts' sums take some
    roundings of 6e-8."""
    g = torch.Generator(DEV).manual_seed(1)
    x = torch.rand(m, k, generator=g, device=DEV)
    w = torch.empty(n, k, dtype=torch.bfloat16, device=DEV)
    for i in range(0, n, 2000):
        w[i:i + 2000].uniform_(0, 1, generator=g)
    wq, xq = fp8.quantize(w, "tiles"), fp8.quantize(x, "rows")
    del w
    xv = xq.dequantize("rows", torch.float32).double()
    wv = wq.dequantize("rows", torch.float32)
    want = torch.cat([xv @ wv[i:i + 2000].double().t() for i in range(0, n, 2000)], 1)
    del wv
    got = fp8.linear(x, wq)
    assert float((got.double() - want).norm() / want.norm()) <= 3.8e-7 + 8 * 6e-8
    y, _ = fp8.forward(x, wq)
    assert torch.equal(y, got)
