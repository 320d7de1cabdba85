"""Refusals of orthogonalised updates, before anything is launched."""

import ctypes

import pytest
import torch

from test_host_device_checks import fake


@pytest.fixture(scope="module")
def abi():
    from block_wise_dynamic_gb300 import build

    build.build()
    from block_wise_dynamic_gb300 import _abi

    return _abi


P = 1 << 20


def i64(*v):
    return (ctypes.c_int64 * len(v))(*v)


def ptrs(*v):
    return (ctypes.c_void_p * len(v))(*v)


def test_orthogonalize_refuses(abi):
    lib = abi.load()
    good = dict(count=2, g=ptrs(P, P), dtype=0, rows=i64(3, 4), cols=i64(5, 6), steps=5, out=ptrs(P, P), work=P, stream=None)
    bad = [dict(count=-1), dict(dtype=9), dict(steps=0), dict(steps=101), dict(g=None), dict(out=None), dict(rows=None), dict(rows=i64(-1, 4)),
           dict(cols=i64(5, 65537)), dict(g=ptrs(P, None)), dict(out=ptrs(None, P)), dict(g=ptrs(P + 2, P)), dict(work=None), dict(work=P + 64)]
    for b in bad:
        assert lib.bwd_orthogonalize(*{**good, **b}.values()) in (1, 2), b
    assert lib.bwd_orthogonalize(*{**good, "count": 0, "work": None}.values()) == 0
    assert lib.bwd_orthogonalize(*{**good, "rows": i64(0, 4), "cols": i64(5, 0), "g": ptrs(None, None), "work": None}.values()) == 0


def test_step_refuses(abi):
    lib = abi.load()

    def hp(**k):
        return ctypes.byref(abi.MuonHParams(**{**dict(lr=0.1, momentum=0.9, weight_decay=0.0, rms=0.2, nesterov=1, steps=5), **k}))

    good = dict(count=1, p=ptrs(P), pt=0, g=ptrs(P), gt=1, m=ptrs(P), rows=i64(3), cols=i64(5), scale=None, hp=hp(), work=P, stream=None)
    nan, inf = float("nan"), float("inf")
    bad = [dict(hp=None), dict(pt=5), dict(gt=5), dict(m=None), dict(m=ptrs(None)), dict(m=ptrs(P + 2)), dict(scale=P + 2)]
    bad += [dict(hp=hp(**k)) for k in (dict(lr=-1.0), dict(lr=nan), dict(lr=inf), dict(momentum=1.0), dict(momentum=-0.1), dict(weight_decay=nan),
                                       dict(rms=-1.0), dict(rms=inf), dict(steps=0))]
    for b in bad:
        assert lib.bwd_muon_step(*{**good, **b}.values()) in (1, 2), b


def test_work_bytes(abi):
    lib = abi.load()
    size = lib.bwd_orthogonalize_work_bytes
    assert size(0, None, None) == 0 and size(-1, None, None) == -1 and size(1, None, i64(1)) == -1
    assert size(1, i64(65537), i64(1)) == -1 and size(2, i64(0, 3), i64(3, 0)) == 0
    one = size(1, i64(100), i64(300))
    # two pairs of 100 x 320 and two of 100 x 128 fp16 values, the norms' parts
    assert one == 2 * 4 * 100 * 320 + 2 * 4 * 100 * 128 + 8 * 512
    assert size(2, i64(100, 300), i64(300, 100)) == 2 * one
    # small matrices of other shapes are worked on together, large ones take turns
    assert size(2, i64(100, 10), i64(300, 10)) == one + 4 * 2560 + 8 * 512
    large = size(1, i64(3000), i64(4000))
    assert size(2, i64(3000, 2000), i64(4000, 3000)) == large == size(3, i64(3000, 100, 2000), i64(4000, 300, 3000))
    # more than a launch takes, in equal parts, with two more pairs of squares, their diagonals and the planes' factors
    assert size(65, i64(*[100] * 65), i64(*[300] * 65)) == 33 * (one + 2 * 4 * 100 * 128) + 13312 + 256


def test_python_refuses():
    from block_wise_dynamic_gb300 import muon

    def f(shape, dtype=torch.float32, index=0):
        return fake(shape, dtype, index)

    with pytest.raises(TypeError):
        muon.orthogonalize([1])
    with pytest.raises(ValueError, match="CUDA"):
        muon.orthogonalize(torch.zeros(2, 2))
    with pytest.raises(TypeError):
        muon.orthogonalize(f((2, 2), torch.float64))
    with pytest.raises(ValueError, match="rows and columns"):
        muon.orthogonalize(f(4))
    p, g, m = f((2, 3)), f((2, 3)), f((2, 3))
    with pytest.raises(ValueError, match="same length"):
        muon.MuonArgs([p], [g, g], [m])
    with pytest.raises(ValueError, match="matrix"):
        muon.MuonArgs([f(6)], [f(6)], [f(6)])
    with pytest.raises(ValueError, match="shape"):
        muon.MuonArgs([p], [f((3, 2))], [m])
    with pytest.raises(TypeError, match="momenta"):
        muon.MuonArgs([p], [g], [f((2, 3), torch.bfloat16)])
    with pytest.raises(ValueError, match="cuda:1"):
        muon.MuonArgs([p], [f((2, 3), index=1)], [m])
    with pytest.raises(TypeError, match="share a dtype"):
        muon.MuonArgs([p, f((2, 3), torch.bfloat16)], [g, g], [m, m])
    for bad in (dict(lr=-1.0), dict(momentum=1.0), dict(weight_decay=-1.0), dict(rms=float("inf")), dict(steps=0)):
        with pytest.raises(ValueError):
            muon.Muon([torch.nn.Parameter(torch.zeros(2, 2))], **bad)
    with pytest.raises(ValueError, match="matrices"):
        muon.Muon([torch.nn.Parameter(torch.zeros(2))])
