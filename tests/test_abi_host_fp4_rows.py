"""The most rows of 4-bit floating point: what is documented passes the checks, one more is refused before a launch."""

import os

import pytest

P = 1 << 20
MOST = 2_097_120


@pytest.fixture(scope="module")
def abi():
    from block_wise_dynamic_gb300 import build

    build.build()
    from block_wise_dynamic_gb300 import _abi

    return _abi


def test_rows(abi):
    lib = abi.load()
    calls = {
        "quantize": lambda rows: lib.bwd_fp4_quantize(P, 1, rows, 10, 10, P, P + 8, None),  # scales off 16 bytes: refused at last
        "dequantize": lambda rows: lib.bwd_fp4_dequantize(P, P + 8, rows, 10, P, 1, None),
        "linear": lambda rows: lib.bwd_fp4_linear(P, 1, rows, 10, 10, P, P + 8, 4, None, P, 4, P, None),
    }
    for name, call in calls.items():
        assert call(MOST) == call(MOST + 1) == 1, name
        message = {}
        for rows in (MOST, MOST + 1):
            call(rows)
            message[rows] = lib.bwd_last_error().decode()
        assert "aligned" in message[MOST] and "65535 * 32 rows" in message[MOST + 1], (name, message)


def test_documents_name_it(abi):
    from block_wise_dynamic_gb300 import fp4

    root = os.path.dirname(os.path.dirname(abi.__file__))
    assert f"{MOST:,} rows" in fp4.__doc__
    with open(os.path.join(root, "include", "bwd.h")) as f:
        assert f"{MOST:,} rows" in f.read()
