"""Layer norm behind a residual update, and its gradients, in float64, from the formulas of include/nvfp4moe.h.

Beside a result, the sum of the absolute values of its terms: what a relative
rounding error of each term is measured against.
"""
import numpy as np


def update(x, residual, scale=1.0):
    """(r', sum of absolute terms)."""
    if residual is None:
        return x, np.abs(x)
    return residual + scale * x, np.abs(residual) + np.abs(scale * x)


def normalized(r, eps):
    """(n, 1 / sqrt(var + eps), the centred row)."""
    c = r - r.mean(1, keepdims=True)
    rho = 1.0 / np.sqrt((c * c).mean(1, keepdims=True) + eps)
    return c * rho, rho, c


def forward(r, w=None, b=None, eps=1e-5):
    n = normalized(r, eps)[0]
    return n * (1.0 if w is None else w) + (0.0 if b is None else b)


def backward(d_y, d_res_out, r, w=None, scale=1.0, eps=1e-5):
    """dict of (gradient, sum of absolute terms): d_residual, d_x, d_w, d_b."""
    n, rho, _ = normalized(r, eps)
    n_abs = np.abs(n) + np.abs(n).mean(1, keepdims=True)
    dn = d_y * (1.0 if w is None else w)
    dr = rho * (dn - dn.mean(1, keepdims=True) - n * (dn * n).mean(1, keepdims=True))
    size = rho * (np.abs(dn) + np.abs(dn).mean(1, keepdims=True) + n_abs * (np.abs(dn) * n_abs).mean(1, keepdims=True))
    if d_res_out is not None:
        dr, size = dr + d_res_out, size + np.abs(d_res_out)
    return {"d_residual": (dr, size), "d_x": (scale * dr, abs(scale) * size),
            "d_w": ((d_y * n).sum(0), (np.abs(d_y) * n_abs).sum(0)), "d_b": (d_y.sum(0), np.abs(d_y).sum(0))}
