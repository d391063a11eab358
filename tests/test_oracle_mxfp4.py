"""The MXFP4 oracle: worked blocks, its rounding against fractions, and what its two scale rules promise (CPU)."""
from fractions import Fraction

import numpy as np
import pytest

import oracle.mxfp4 as MX


def test_worked_block():
    x = np.zeros((1, 32))
    x[0, :9] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.01, 7.9]   # amax in [4, 8): unit 1
    q, s = MX.quantize(x)
    assert q.shape == (1, 64) and s.shape == (1, 1, 4) and s[0, 0].tolist() == [127, 0, 0, 0]
    assert MX.dequantize(q, s)[0, :9].tolist() == [0, 1, 1, 2, 2, 4, 4, -6, 6]
    q, s = MX.quantize(x, MX.CEIL)                                      # 7.9 > 6: unit 2
    assert s[0, 0, 0] == 128 and MX.dequantize(q, s)[0, :9].tolist() == [0, 1, 1, 2, 2, 4, 4, -6, 8]
    assert MX.quantize(np.full((1, 32), 6.0), MX.CEIL)[1][0, 0, 0] == 127
    assert MX.quantize(np.zeros((1, 32)))[1][0, 0, 0] == 0
    assert MX.quantize(np.full((1, 32), 2.0 ** -149))[1][0, 0, 0] == 0
    x[0, 3] = np.inf
    assert MX.quantize(x)[1][0, 0].tolist() == [255, 0, 0, 0] and np.isnan(MX.dequantize(*MX.quantize(x))[0, :32]).all()


@pytest.mark.parametrize("rule", [MX.FLOOR, MX.CEIL])
def test_nearest_of_all(rule):
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((6, 100)) * np.exp2(rng.integers(-130, 120, (6, 1)))).astype(np.float32).astype(np.float64)
    q, s = MX.quantize(x, rule)
    v = MX.dequantize(q, s)
    assert not v[:, 100:].any()
    for i in range(6):
        for j in range(100):
            unit = Fraction(2) ** (int(s[j // 128, i, (j // 32) % 4]) - 127)
            err = abs(Fraction(float(v[i, j])) - Fraction(float(x[i, j])))
            assert err == min(abs(abs(Fraction(float(x[i, j]))) - Fraction(float(m)) * unit) for m in MX.VALUES)
        for b in range(4):
            top = np.abs(x[i, 32 * b:32 * b + 32]).max()
            unit = 2.0 ** (int(s[0, i, b]) - 127)
            if s[0, i, b] > 0:
                assert (top <= 6 * unit and top > 3 * unit) if rule == MX.CEIL else 4 * unit <= top < 8 * unit
