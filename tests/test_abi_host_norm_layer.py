"""Refusals of the layer norm, before anything is launched."""

import ctypes

import pytest
import torch

from test_host_device_checks import fake


@pytest.fixture(scope="module")
def lib():
    from block_wise_dynamic_gb300 import build

    build.build()
    from block_wise_dynamic_gb300 import _abi

    return _abi.load()


def test_forward_refuses(lib):
    p = ctypes.c_void_p(1 << 20)
    good = dict(x=p, dtype=1, rows=3, width=10, ldx=10, gamma=p, beta=p, vectors=0, eps=1e-5, y=p, mean=p, rstd=p, stream=None)
    bad = [dict(dtype=7), dict(vectors=2), dict(rows=-1), dict(width=0), dict(width=16385), dict(ldx=9), dict(eps=-1.0), dict(eps=float("nan")),
           dict(x=None), dict(y=None), dict(x=ctypes.c_void_p((1 << 20) + 1)), dict(gamma=ctypes.c_void_p((1 << 20) + 2)),
           dict(mean=ctypes.c_void_p((1 << 20) + 2))]
    for b in bad:
        assert lib.bwd_norm_forward(*{**good, **b}.values()) in (1, 2), b
    assert lib.bwd_norm_forward(*{**good, "rows": 0, "x": None, "y": None}.values()) == 0


def test_backward_refuses(lib):
    p = ctypes.c_void_p(1 << 20)
    good = dict(dy=p, x=p, dtype=1, rows=3, width=10, lddy=10, ldx=10, gamma=p, vectors=0, mean=p, rstd=p, dx=p, dgamma=p, dbeta=p, work=p,
                stream=None)
    bad = [dict(dtype=-1), dict(vectors=2), dict(rows=-1), dict(width=0), dict(width=16385), dict(lddy=9), dict(ldx=9), dict(dy=None),
           dict(x=None), dict(mean=None), dict(rstd=None), dict(work=None), dict(dx=ctypes.c_void_p((1 << 20) + 1)),
           dict(dgamma=ctypes.c_void_p((1 << 20) + 2)), dict(work=ctypes.c_void_p((1 << 20) + 2))]
    for b in bad:
        assert lib.bwd_norm_backward(*{**good, **b}.values()) in (1, 2), b
    assert lib.bwd_norm_backward(*{**good, "dx": None, "dgamma": None, "dbeta": None}.values()) == 0


def test_work_bytes(lib):
    assert lib.bwd_norm_backward_work_bytes(-1, 10) == -1 and lib.bwd_norm_backward_work_bytes(1, 16385) == -1
    assert lib.bwd_norm_backward_work_bytes(0, 100) == 0
    for rows in (1, 7, 8, 9, 1000, 1 << 20):
        for width in (1, 512, 513, 8192, 8193, 16384):
            parts = lib.bwd_norm_backward_work_bytes(rows, width) // (8 * width)
            assert 1 <= parts <= min(rows, 160 * 16)


def test_python_refuses():
    from block_wise_dynamic_gb300 import norm

    x = fake((4, 8), torch.bfloat16, 0)
    v = fake(8, torch.float32, 0)
    r = fake(4, torch.float32, 0)
    with pytest.raises(ValueError, match="cuda:1"):
        norm.forward(x, fake(8, torch.float32, 1))
    with pytest.raises(TypeError, match="float32 or of x's"):
        norm.forward(x, fake(8, torch.float16, 0))
    with pytest.raises(TypeError, match="beta"):
        norm.forward(x, v, fake(8, torch.bfloat16, 0))
    with pytest.raises(ValueError, match="8 elements"):
        norm.forward(x, fake(7, torch.float32, 0))
    with pytest.raises(ValueError, match="last dimension"):
        norm.forward(fake((4, 16385), torch.float32, 0))
    with pytest.raises(ValueError, match="CUDA"):
        norm.forward(torch.zeros(4, 8))
    with pytest.raises(TypeError):
        norm.forward(fake((4, 8), torch.float64, 0))
    with pytest.raises(ValueError, match="dy"):
        norm.backward(fake((4, 8), torch.float32, 0), x, v, r, r)
    with pytest.raises(ValueError, match="dy"):
        norm.backward(fake((4, 8), torch.bfloat16, 1), x, v, r, r)
    with pytest.raises(ValueError, match="mean"):
        norm.backward(x, x, v, fake(3, torch.float32, 0), r)
    with pytest.raises(ValueError, match="dim must"):
        norm.LayerNorm(0, device="cpu")
