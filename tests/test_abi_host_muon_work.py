"""The limit of the workspace of orthogonalised updates, before anything is launched."""

import ctypes

import pytest
import torch

from test_abi_host_muon import P, i64, ptrs
from test_host_device_checks import fake


@pytest.fixture(scope="module")
def abi():
    from block_wise_dynamic_gb300 import build

    build.build()
    from block_wise_dynamic_gb300 import _abi

    return _abi


def test_work_bytes_within_a_limit(abi):
    lib = abi.load()
    size = lib.bwd_muon_work_bytes
    rows, cols = i64(*[1024] * 48), i64(*[4096] * 48)
    whole, one = lib.bwd_orthogonalize_work_bytes(48, rows, cols), size(1, rows, cols, 0)
    # two pairs of 1024 x 4096 and four of 1024 x 1024 fp16 values, 50 MB, to a matrix
    assert one >= 8 * 1024 * 4096 + 16 * 1024 * 1024 and whole == size(48, rows, cols, 0) == size(48, rows, cols, 4 << 30) > 47 * one
    assert whole < 4 << 30
    for limit in (2 << 30, 1 << 30, 100 << 20, one):
        assert one <= size(48, rows, cols, limit) <= limit
    assert size(48, rows, cols, 1) == one  # a matrix takes what it takes
    # small ones, which share their launches, too
    rows, cols = i64(*range(20, 36)), i64(*[90] * 16)
    alone = max(size(1, i64(r), i64(90), 0) for r in range(20, 36))
    assert size(16, rows, cols, 0) > 7 * alone // 2
    assert size(16, rows, cols, 3 * alone) <= 3 * alone and size(16, rows, cols, 1) == alone
    assert size(1, rows, cols, -1) == -1 and size(0, None, None, 5) == 0


def test_a_negative_limit_is_refused(abi):
    lib = abi.load()
    hp = abi.MuonHParams(0.1, 0.9, 0.0, 0.2, 1, 5, -1)
    assert lib.bwd_muon_step(1, ptrs(P), 0, ptrs(P), 1, ptrs(P), i64(3), i64(5), None, ctypes.byref(hp), P, None) in (1, 2)


def test_python_refuses():
    from block_wise_dynamic_gb300 import muon

    p = fake((2, 3), torch.float32, 0)
    for bad in (0, -5, 1 << 63):
        with pytest.raises(ValueError, match="work_bytes"):
            muon.MuonArgs([p], [p], [p], work_bytes=bad)
        with pytest.raises(ValueError, match="work_bytes"):
            muon.Muon([torch.nn.Parameter(torch.zeros(2, 2))], work_bytes=bad)
