"""Refusals and sizes of 4-bit floating point, before anything is launched."""

import pytest
import torch

from test_host_device_checks import fake


@pytest.fixture(scope="module")
def lib():
    from block_wise_dynamic_gb300 import build

    build.build()
    from block_wise_dynamic_gb300 import _abi

    return _abi.load()


P = 1 << 20


def test_sizes(lib):
    from block_wise_dynamic_gb300 import fp4

    assert lib.bwd_fp4_pitch(-1) == -1 and lib.bwd_fp4_scale_bytes(1, -1) == -1 and lib.bwd_fp4_linear_work_bytes(-1, 1) == -1
    for cols in (0, 1, 2, 31, 32, 33, 127, 128, 129, 130, 255, 256, 257, 4096, 11008):
        pitch = lib.bwd_fp4_pitch(cols)
        assert 2 * pitch >= cols and pitch % 16 == 0 and (pitch % 128 == 0 or pitch <= 64)
        for rows in (0, 1, 127, 128, 129, 1000):
            layout = fp4._layout(rows, cols)
            assert layout[0] == pitch and layout[2] - layout[1] == lib.bwd_fp4_scale_bytes(rows, cols)
            assert fp4._work(rows, cols) == lib.bwd_fp4_linear_work_bytes(rows, cols)
    for rows, cols in ((8, 229_376), (8, 229_377), (9, 1), (1, 1 << 20)):
        assert fp4._work(rows, cols) == lib.bwd_fp4_linear_work_bytes(rows, cols)
        assert (fp4._work(rows, cols) == 0) == (rows <= 8 and cols <= 229_376)


def test_quantize_and_dequantize_refuse(lib):
    good = dict(x=P, dtype=1, rows=3, cols=10, ld=10, codes=P, scales=P, stream=None)
    for b in (dict(dtype=5), dict(rows=-1), dict(cols=-1), dict(cols=(1 << 30) + 1), dict(rows=65535 * 32 + 1), dict(ld=9), dict(x=None), dict(x=P + 1),
              dict(codes=None), dict(scales=None), dict(codes=P + 8), dict(scales=P + 4)):
        assert lib.bwd_fp4_quantize(*{**good, **b}.values()) in (1, 2), b
    good = dict(codes=P, scales=P, rows=3, cols=10, out=P, dtype=0, stream=None)
    for b in (dict(dtype=5), dict(rows=-1), dict(out=None), dict(out=P + 2), dict(codes=None), dict(scales=P + 4)):
        assert lib.bwd_fp4_dequantize(*{**good, **b}.values()) in (1, 2), b


def test_products_refuse(lib):
    good = dict(m=3, n=4, k=10, a=P, sa=P, b=P, sb=P, bias=P, out=P, ldo=4, dtype=1, stream=None)
    for b in (dict(dtype=5), dict(m=-1), dict(k=(1 << 30) + 1), dict(ldo=3), dict(out=None), dict(out=P + 1), dict(bias=P + 1), dict(a=None),
              dict(sb=None), dict(b=P + 8), dict(sa=P + 8)):
        assert lib.bwd_fp4_matmul(*{**good, **b}.values()) in (1, 2), b
    good = dict(x=P, dtype=1, rows=3, cols=10, ld=10, w=P, ws=P, n=4, bias=P, y=P, ldy=4, work=P, stream=None)
    for b in (dict(dtype=5), dict(rows=-1), dict(ld=9), dict(n=-1), dict(ldy=3), dict(x=None), dict(w=None), dict(ws=None), dict(y=None),
              dict(rows=9, work=None), dict(work=P + 8), dict(w=P + 8), dict(y=P + 1), dict(bias=P + 1)):
        assert lib.bwd_fp4_linear(*{**good, **b}.values()) in (1, 2), b


def test_python_refuses():
    from block_wise_dynamic_gb300 import fp4

    def f(shape, dtype=torch.bfloat16, index=0):
        return fake(shape, dtype, index)

    def matrix(rows, cols, index=0):
        return fp4.Fp4Matrix(rows, cols, torch.bfloat16, f(fp4._layout(rows, cols)[2], torch.uint8, index))

    w = matrix(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        fp4.quantize(torch.zeros(2, 2))
    with pytest.raises(TypeError):
        fp4.quantize(f((2, 2), torch.float64))
    with pytest.raises(TypeError, match="Fp4Matrix"):
        fp4.linear(f((2, 8)), f((4, 8)))
    with pytest.raises(ValueError, match="last dimension"):
        fp4.linear(f((2, 9)), w)
    with pytest.raises(ValueError, match="cuda:0"):
        fp4.linear(f((2, 8), index=1), w)
    with pytest.raises(TypeError, match="bias"):
        fp4.linear(f((2, 8)), w, f(4, torch.float32))
    with pytest.raises(ValueError, match="4 elements"):
        fp4.linear(f((2, 8)), w, f(5))
    with pytest.raises(ValueError, match="9 elements, b.s 8"):
        fp4.matmul(matrix(2, 9), w)
    with pytest.raises(ValueError, match="cuda:1"):
        fp4.matmul(matrix(2, 8), matrix(4, 8, 1))
    with pytest.raises(TypeError, match="dtype"):
        fp4.dequantize(w, torch.float64)
    with pytest.raises(ValueError, match="elements"):
        fp4.Fp4Matrix(4, 8, torch.bfloat16, f(16, torch.uint8))
