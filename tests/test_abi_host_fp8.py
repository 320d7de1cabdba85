"""The 8-bit floating point, 32-bit-state and norm entry points refuse bad
arguments on the host, before anything touches a GPU, and their size helpers
agree with the Python binding's."""

import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from block_wise_dynamic_gb300 import build as b

    b.build()
    from block_wise_dynamic_gb300 import _abi

    return _abi.load()


FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: refused first
ODD = ctypes.c_void_p(0x1001)
OK, INVALID, UNSUPPORTED = 0, 1, 2


def test_size_helpers(lib):
    from block_wise_dynamic_gb300 import fp8

    for n in (0, 1, 15, 16, 17, 512, 513, 640, 4097, 1 << 30):
        assert lib.bwd_fp8_pitch(n) == fp8._pitch(n) >= n and fp8._pitch(n) % 16 == 0
        for k in (0, 1, 127, 128, 129, 512, 513, 11008):
            assert lib.bwd_fp8_scale_bytes(n, k) == fp8._scale_bytes(n, k)
    assert lib.bwd_fp8_pitch(-1) == lib.bwd_fp8_pitch((1 << 30) + 1) == -1
    assert lib.bwd_fp8_scale_bytes(-1, 5) == lib.bwd_fp8_scale_bytes(5, 1 << 31) == -1
    for rows in (0, 1, 16, 17, 300):
        for k in (1, 4096, 1003):
            codes = fp8._round256(rows * fp8._pitch(k)) + fp8._round256(fp8._scale_bytes(rows, k))
            assert lib.bwd_fp8_linear_work_bytes(rows, k) == (0 if rows <= fp8._FUSED_ROWS else codes)
            both = codes + fp8._round256(rows * fp8._pitch(k)) + fp8._round256(fp8._scale_bytes(k, rows))
            assert lib.bwd_fp8_linear_backward_work_bytes(rows, k) == both + fp8._round256((rows + 127) // 128 * k * 4)
    assert lib.bwd_fp8_linear_work_bytes(-1, 1) == lib.bwd_fp8_linear_backward_work_bytes(1, -1) == -1
    assert lib.bwd_grad_norm_work_bytes(-1) == -1 and lib.bwd_grad_norm_work_bytes(0) >= 16


def test_quantize_refusals(lib):
    def q(x=FAKE, dtype=1, rows=4, cols=8, ld=8, blocks=1, rc=FAKE, rs=FAKE, cc=None, cs=None, sums=None, work=None):
        return lib.bwd_fp8_quantize(x, dtype, rows, cols, ld, blocks, rc, rs, cc, cs, sums, work, None)

    assert q(dtype=7) == UNSUPPORTED
    assert q(rows=-1) == q(cols=-1) == q(ld=7) == q(blocks=0) == q(blocks=5) == q(blocks=8) == INVALID
    assert q(rows=65535 * 128 + 1) == INVALID
    assert q(x=None) == q(rc=None) == q(rs=None) == q(x=ODD) == q(rc=ODD) == INVALID
    assert q(blocks=2, rc=None, rs=None) == q(blocks=3) == q(blocks=4) == INVALID
    assert q(sums=FAKE, work=FAKE) == INVALID          # sums need column blocks
    assert q(blocks=2, cc=FAKE, cs=FAKE, sums=FAKE) == q(blocks=2, cc=FAKE, cs=FAKE, sums=ODD, work=FAKE) == INVALID
    assert q(cols=0) == OK and q(rows=0, x=None, rc=None, rs=None) == OK


def test_dequantize_and_matmul_refusals(lib):
    assert lib.bwd_fp8_dequantize(FAKE, FAKE, 1, 2, 2, FAKE, 9, None) == UNSUPPORTED
    assert lib.bwd_fp8_dequantize(FAKE, None, 1, 2, 2, FAKE, 0, None) == INVALID
    assert lib.bwd_fp8_dequantize(FAKE, FAKE, 1, -2, 2, FAKE, 0, None) == INVALID
    assert lib.bwd_fp8_dequantize(FAKE, FAKE, 1, 2, 2, ODD, 0, None) == INVALID
    assert lib.bwd_fp8_dequantize(None, None, 1, 0, 2, None, 0, None) == OK

    def mm(m=4, n=4, k=4, a=FAKE, sa=FAKE, b=FAKE, sb=FAKE, bias=None, out=FAKE, ldo=4, dtype=1):
        return lib.bwd_fp8_matmul(m, n, k, a, 0, sa, b, 0, sb, bias, out, ldo, dtype, None)

    assert mm(dtype=3) == UNSUPPORTED
    assert mm(m=-1) == mm(k=-1) == mm(ldo=3) == mm(n=1 << 31, ldo=1 << 31) == INVALID
    assert mm(a=None) == mm(sa=None) == mm(b=None) == mm(sb=None) == mm(out=None) == INVALID
    assert mm(a=ODD) == mm(sb=ODD) == mm(out=ODD) == mm(bias=ODD) == INVALID
    assert mm(m=0, out=None) == OK and mm(n=0, ldo=0, out=None) == OK


def test_linear_refusals(lib):
    def fwd(x=FAKE, dtype=1, rows=40, cols=8, ld=8, w=FAKE, ws=FAKE, n=4, bias=None, y=FAKE, ldy=4, cc=None, cs=None, work=FAKE):
        return lib.bwd_fp8_linear(x, dtype, rows, cols, ld, w, ws, n, bias, y, ldy, cc, cs, work, None)

    assert fwd(dtype=-1) == UNSUPPORTED
    assert fwd(rows=-1) == fwd(ld=7) == fwd(ldy=3) == fwd(n=-1) == INVALID
    assert fwd(x=None) == fwd(w=None) == fwd(ws=None) == fwd(y=None) == fwd(work=None) == fwd(cc=FAKE) == INVALID
    assert fwd(w=ODD) == fwd(y=ODD) == fwd(bias=ODD) == fwd(work=ODD) == INVALID

    def bwd(dy=FAKE, dtype=1, rows=40, n=4, ld=4, w=FAKE, ws=FAKE, xc=FAKE, xs=FAKE, k=8, dx=FAKE, lddx=8, dw=FAKE, lddw=8, db=None, work=FAKE):
        return lib.bwd_fp8_linear_backward(dy, dtype, rows, n, ld, w, ws, xc, xs, k, dx, lddx, dw, lddw, db, work, None)

    assert bwd(dtype=3) == UNSUPPORTED
    assert bwd(rows=-1) == bwd(ld=3) == bwd(k=-1) == bwd(lddx=7) == bwd(lddw=7) == INVALID
    assert bwd(dy=None) == bwd(w=None) == bwd(ws=None) == bwd(xc=None) == bwd(xs=None) == bwd(work=None) == INVALID
    assert bwd(dx=ODD) == bwd(dw=ODD) == bwd(db=ODD) == bwd(w=ODD) == bwd(work=ODD) == INVALID
    assert bwd(dx=None, dw=None) == OK


def test_adam32_and_norm_refusals(lib):
    from block_wise_dynamic_gb300._abi import AdamWHParams

    one = (ctypes.c_void_p * 1)(0x1000)
    odd = (ctypes.c_void_p * 1)(0x1001)
    n1, neg = (ctypes.c_int64 * 1)(4), (ctypes.c_int64 * 1)(-4)
    good = AdamWHParams(1e-3, 0.9, 0.999, 1e-8, 0.0, 1)

    def step(T=1, p=one, pd=0, g=one, gd=0, m=one, v=one, n=n1, scale=None, hp=good):
        return lib.bwd_adam32_step_multi(T, p, pd, g, gd, m, v, n, scale, None if hp is None else ctypes.byref(hp), None)

    assert step(pd=5) == step(gd=5) == UNSUPPORTED
    assert step(T=-1) == step(p=None) == step(n=None) == step(n=neg) == step(hp=None) == step(scale=ODD) == INVALID
    assert step(p=odd) == step(g=odd, gd=1) == step(m=odd) == step(v=(ctypes.c_void_p * 1)(None)) == INVALID
    for bad in (dict(step=0), dict(lr=float("nan")), dict(beta2=1.0), dict(eps=-1.0), dict(weight_decay=-1.0)):
        hp = AdamWHParams(1e-3, 0.9, 0.999, 1e-8, 0.0, 1)
        for k, x in bad.items():
            setattr(hp, k, x)
        assert step(hp=hp) == INVALID
    assert step(T=0) == OK

    t0, t9 = (ctypes.c_int32 * 1)(0), (ctypes.c_int32 * 1)(9)

    def norm(T=1, g=one, types=t0, n=n1, top=1.0, scale=1.0, f=FAKE, out=FAKE, work=FAKE):
        return lib.bwd_grad_norm(T, g, types, n, top, scale, f, out, work, None)

    assert norm(types=t9) == UNSUPPORTED
    assert norm(T=-1) == norm(g=None) == norm(types=None) == norm(n=None) == norm(n=neg) == norm(g=odd) == INVALID
    assert norm(top=0.0) == norm(top=float("nan")) == norm(scale=0.0) == norm(scale=float("inf")) == norm(scale=1e-45) == INVALID
    assert norm(f=None) == norm(out=None) == norm(work=None) == norm(f=ODD) == norm(work=ODD) == INVALID
