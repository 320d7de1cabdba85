"""The steps with a count in device memory refuse bad arguments on the host."""

import ctypes

import pytest

FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: refused first
ODD = ctypes.c_void_p(0x1004)   # no multiple of 8
OK, INVALID, UNSUPPORTED = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    from block_wise_dynamic_gb300 import build as b

    b.build()
    from block_wise_dynamic_gb300 import _abi

    return _abi.load()


one, odd, none = (ctypes.c_void_p * 1)(0x1000), (ctypes.c_void_p * 1)(0x1001), (ctypes.c_void_p * 1)(None)
n1, neg = (ctypes.c_int64 * 1)(4), (ctypes.c_int64 * 1)(-4)


def test_32_bit_states(lib):
    from block_wise_dynamic_gb300._abi import AdamWHParams

    def step(T=1, p=one, pd=0, g=one, gd=0, m=one, v=one, n=n1, scale=None, count=FAKE, **hp):
        h = AdamWHParams(*{**dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=0), **hp}.values())
        return lib.bwd_adam32_step_multi_counted(T, p, pd, g, gd, m, v, n, scale, count, ctypes.byref(h), None)

    assert step(count=None) == step(count=ODD) == step(T=-1) == step(p=none) == step(m=odd) == step(n=neg) == INVALID
    assert step(scale=ctypes.c_void_p(0x1002)) == step(beta1=1.0) == step(eps=-1.0) == step(lr=float("inf")) == INVALID
    assert step(pd=9) == step(gd=9) == UNSUPPORTED
    assert step(T=0) == OK
    assert lib.bwd_adam32_step_multi_counted(1, one, 0, one, 0, one, one, n1, None, FAKE, None, None) == INVALID


def test_8_bit_states(lib):
    from block_wise_dynamic_gb300._abi import AdamHParams

    def step(T=1, p=one, pd=0, g=one, gd=0, mc=one, ma=one, vc=one, va=one, n=n1, scale=None, count=FAKE, **hp):
        h = AdamHParams(*{**dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=0), **hp}.values())
        return lib.bwd_adam8bit_step_multi_counted(T, p, pd, g, gd, mc, ma, vc, va, n, scale, count, ctypes.byref(h), None)

    assert step(count=None) == step(count=ODD) == step(T=-1) == step(mc=none) == step(ma=odd) == step(n=neg) == INVALID
    assert step(scale=ctypes.c_void_p(0x1002)) == step(beta2=1.0) == step(weight_decay=-1.0) == INVALID
    assert step(pd=9) == step(gd=9) == UNSUPPORTED
    assert step(T=0) == OK
    assert lib.bwd_adam8bit_step_multi_counted(1, one, 0, one, 0, one, one, one, one, n1, None, FAKE, None, None) == INVALID
