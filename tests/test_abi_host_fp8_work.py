"""The forward pass's workspace around the sizes that need none."""


def test_linear_work_bytes():
    from block_wise_dynamic_gb300 import build as b

    b.build()
    from block_wise_dynamic_gb300 import _abi, fp8

    lib = _abi.load()
    for rows in (0, 1, 16, 17):
        for cols in (1, 4096, fp8._FUSED_COLS, fp8._FUSED_COLS + 1, 1 << 20):
            codes = fp8._round256(rows * fp8._pitch(cols)) + fp8._round256(fp8._scale_bytes(rows, cols))
            want = 0 if rows <= 16 and cols <= 245_760 else codes
            assert lib.bwd_fp8_linear_work_bytes(rows, cols) == fp8._forward_work(rows, cols) == want
