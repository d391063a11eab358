"""The slopes of the gate's pointwise scores in the oracle, also where a score is 1 to float64's last bit."""
from fractions import Fraction
import math

import numpy as np
import pytest

import oracle.gate as G


@pytest.mark.parametrize("x", [-300.0, -40.0, -1.0, 0.0, 0.5, 20.0, 33.25, 36.5, 60.0, 300.0])
def test_sigmoid_slope(x):
    e = Fraction(math.exp(-abs(x)))          # half a step of float64 away from e^-|x|; all that follows is exact
    want = e / (1 + e) ** 2
    got = Fraction(float(G.score_slopes(np.array([x]), G.SIGMOID)[0]))
    assert abs(got - want) <= want * Fraction(8, 2 ** 53)


def test_no_slope_where_nothing_can_be_chosen():
    assert not G.score_slopes(np.array([-np.inf]), G.SIGMOID).any()
    assert not G.score_slopes(np.array([-np.inf]), G.SQRT_SOFTPLUS).any()
