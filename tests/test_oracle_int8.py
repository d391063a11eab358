"""The int8 oracle: worked values and the error bound of its rounding (CPU)."""
from fractions import Fraction

import numpy as np

import oracle.int8 as I8


def test_worked_rows():
    x = np.array([[127.0, 0.5, 1.5, -2.5, -127.0, 63.5], [0.0] * 6, [1.0, 0.5, -0.25, 1 / 127, 0.0, -1.0]])
    q, s = I8.quantize_rows(x)
    assert q[0].tolist() == [127, 0, 2, -2, -127, 64] and s[0] == 1.0
    assert not q[1].any() and s[1] == 0.0
    # 0.5 / RN(1 / 127) lies just off 63.5, on the side that the rounding of the scale leaves
    side = Fraction(1, 2) / Fraction(float(s[2])) > Fraction(127, 2)
    assert q[2, 1] == (64 if side else 63) and q[2, 0] == 127 and q[2, 5] == -127


def test_half_a_step():
    x = np.random.default_rng(1).standard_normal((50, 64)) * np.logspace(-6, 6, 50)[:, None]
    x = x.astype(np.float32).astype(np.float64)
    q, s = I8.quantize_rows(x)
    # half a step, and where the scale was rounded down the largest element up to 127 * 2^-24 steps more
    assert (np.abs(q * s.astype(np.float64)[:, None] - x) <= s[:, None] * (0.5 + 1e-5)).all()
