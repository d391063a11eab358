"""Microscaled 4-bit floats: blocks of 32 E2M1 values and a power of two, in float64 (every step exact)."""
import numpy as np

VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
FLOOR, CEIL = 0, 1


def nearest(a):
    """Index of the magnitude nearest to a >= 0, ties to the even index: by distance, whatever the grid."""
    d = np.abs(a[..., None] - VALUES)
    best = d.min(-1, keepdims=True)
    near = d == best                       # one index, or two next to each other
    order = np.where(near, np.arange(8) % 2, 2)
    return order.argmin(-1).astype(np.uint8)


def exponents(amax, rule):
    """The block's power of two for its largest magnitude, at least -127."""
    m, e = np.frexp(amax)                  # amax = m 2^e, m in [1/2, 1)
    p = e - 3                              # floor(log2 amax) - 2
    if rule == CEIL:
        p = p + (amax > 6.0 * np.exp2(p.astype(np.float64)))
    return np.where(amax > 0, np.maximum(p, -127), -127)


def quantize(x, rule=FLOOR):
    """x float64 [M, K] -> (q uint8 [M, Kp / 2], scale uint8 [Kp / 128, M, 4]) with K padded to whole groups of 128."""
    x = np.asarray(x, np.float64)
    M, K = x.shape
    by = np.zeros((M, -(-K // 128) * 128))
    by[:, :K] = x
    by = by.reshape(M, -1, 32)
    whole = np.isfinite(by).all(-1)
    amax = np.abs(np.where(np.isfinite(by), by, 0)).max(-1)
    e = exponents(amax, rule)
    v = np.where(whole[..., None], by, 0) / np.exp2(e.astype(np.float64))[..., None]
    nib = nearest(np.abs(v)) | (np.signbit(v).astype(np.uint8) << 3)
    nib = nib.reshape(M, -1)
    code = np.where(whole, e + 127, 255).astype(np.uint8)
    return nib[:, 0::2] | (nib[:, 1::2] << 4), np.ascontiguousarray(code.reshape(M, -1, 4).transpose(1, 0, 2))


def dequantize(q, scale):
    """float64 [R, K] of the values; NaN where the scale is 255."""
    nib = np.stack([q & 15, q >> 4], -1).reshape(q.shape[0], -1)
    v = VALUES[nib & 7] * np.where(nib > 7, -1.0, 1.0)
    code = scale.transpose(1, 0, 2).reshape(q.shape[0], -1)
    s = np.where(code == 255, np.nan, np.exp2(code.astype(np.float64) - 127))
    return v * np.repeat(s, 32, axis=1)
