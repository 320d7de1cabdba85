"""The 64-bit statement of microscaled 4-bit floating point."""

import numpy as np
import pytest

from oracle import fp4 as ref


def test_rounding():
    # each value stays, each midpoint goes to the even code
    assert (ref.round_code(ref.GRID) == np.arange(8)).all()
    middle = (ref.GRID[1:] + ref.GRID[:-1]) / 2
    assert ref.round_code(middle).tolist() == [0, 2, 2, 4, 4, 6, 6]
    assert (ref.round_code(middle * (1 - 1e-15)) == np.arange(7)).all()
    assert (ref.round_code(-middle * (1 + 1e-15)) == np.arange(1, 8)).all()


@pytest.mark.parametrize("a,e", [(6.0, 0), (np.nextafter(6.0, 7), 1), (3.0, -1), (4.0, 0), (12.0, 1), (0.0, -127), (2.0 ** -149, -127),
                                 (3.4028234663852886e38, 126), (1.5 * 2.0 ** 100, 98), (1.25 * 2.0 ** 100, 98), (1.75 * 2.0 ** 100, 99)])
def test_exponents(a, e):
    assert ref.exponent(a) == e


def test_blocks():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 70)) * np.exp(3 * rng.standard_normal((3, 70)))
    x[1, 40] = np.inf
    q, e = ref.quantize(x)
    assert e.shape == (3, 3) and np.isnan(q[1, 32:64]).all() and np.isfinite(q[1, :32]).all()
    for b in range(3):
        part, top = x[0, 32 * b:32 * b + 32], np.abs(x[0, 32 * b:32 * b + 32]).max()
        s = 2.0 ** e[0, b]
        assert 3 * s < top <= 6 * s
        # no farther than half of the step around a value: 1 at most from 4 on, a quarter below 2
        assert (np.abs(q[0, 32 * b:32 * b + 32] - part) <= s * np.where(np.abs(part) > 4 * s, 1, np.where(np.abs(part) > 2 * s, .5, .25))).all()
    assert np.array_equal(ref.quantize(q[:1])[0], q[:1])
