"""8-bit integer rows and their products, exactly (float64, and fractions where float64 would decide a tie)."""
from fractions import Fraction

import numpy as np


def quantize_rows(x):
    """x float64 [M, K] -> (q int8, scale float32): scale = RN_f32(amax * RN_f32(1 / 127)), q = rne(x / scale)."""
    x = np.asarray(x, np.float64)
    s = (np.abs(x).max(1).astype(np.float32) * (np.float32(1) / np.float32(127))).astype(np.float32)
    d = np.where(s > 0, s, 1).astype(np.float64)[:, None]
    q = np.rint(x / d)
    # x / d in float64 may land on a half that the real quotient only comes close to: as a fraction it is exact
    for i, j in zip(*np.nonzero(np.floor(x / d) + 0.5 == x / d)):
        q[i, j] = round(Fraction(float(x[i, j])) / Fraction(float(d[i, 0])))
    return np.where(s[:, None] > 0, np.clip(q, -127, 127), 0).astype(np.int8), s


def gemm(a_q, a_s, b_q, b_s):
    """float64 [M, N]: the integer sums are below 2^53, so float64 holds them."""
    return (a_q.astype(np.float64) @ b_q.astype(np.float64).T) * a_s.astype(np.float64)[:, None] * b_s.astype(np.float64)


def silu_mul(g, u):
    return g / (1.0 + np.exp(-np.clip(g, -700, None))) * u
