"""The norms around the expert FFN and their gradients, in float64, from the formulas of include/nvfp4moe.h.

Every function also returns, beside each result, the sum of the absolute
values of its terms: what a relative rounding error of each term is measured
against.
"""
import numpy as np


def _col(gate):
    return 1.0 if gate is None else np.asarray(gate, np.float64)


def branch(x, w_post, gate, scale, eps):
    """scale * gate * n."""
    x = np.asarray(x, np.float64)
    n = x if w_post is None else x / np.sqrt((x * x).mean(1, keepdims=True) + eps) * w_post
    return scale * _col(gate) * n


def update(x, residual, w_post=None, gate=None, scale=1.0, eps=1e-6):
    """(r', sum of absolute terms)."""
    b = branch(x, w_post, gate, scale, eps)
    r = np.zeros_like(b) if residual is None else np.asarray(residual, np.float64)
    return r + b, np.abs(r) + np.abs(b)


def normalize(r, w_pre, eps=1e-6):
    r = np.asarray(r, np.float64)
    return r / np.sqrt((r * r).mean(1, keepdims=True) + eps) * w_pre


def backward(d_y, d_res_out, x, res_out, w_pre=None, w_post=None, gate=None, scale=1.0, eps=1e-6):
    """dict of (gradient, sum of absolute terms)."""
    x, r = np.asarray(x, np.float64), np.asarray(res_out, np.float64)
    dr = np.zeros_like(r) if d_res_out is None else np.asarray(d_res_out, np.float64)
    dr_abs = np.abs(dr)
    out = {}
    if w_pre is not None:
        rho = 1.0 / np.sqrt((r * r).mean(1, keepdims=True) + eps)
        rn, dn = r * rho, np.asarray(d_y, np.float64) * w_pre
        out["d_w_pre"] = ((d_y * rn).sum(0), np.abs(d_y * rn).sum(0))
        dr = dr + rho * (dn - rn * (dn * rn).mean(1, keepdims=True))
        dr_abs = dr_abs + rho * (np.abs(dn) + np.abs(rn) * np.abs(dn * rn).mean(1, keepdims=True))
    out["d_residual"] = (dr, dr_abs)
    sig = 1.0 / np.sqrt((x * x).mean(1, keepdims=True) + eps)
    xn = x * sig if w_post is not None else x
    wp = 1.0 if w_post is None else w_post
    db, db_abs = scale * dr, abs(scale) * dr_abs
    if gate is not None:
        axis = 0 if np.asarray(gate).ndim == 1 else 1
        dg, dg_abs = (db * xn * wp).sum(axis), (db_abs * np.abs(xn * wp)).sum(axis)
        out["d_gate"] = (dg, dg_abs) if axis == 0 else (dg[:, None], dg_abs[:, None])
    db, db_abs = db * _col(gate), db_abs * np.abs(_col(gate))
    if w_post is not None:
        out["d_w_post"] = ((db * xn).sum(0), (db_abs * np.abs(xn)).sum(0))
        dxn, dxn_abs = db * wp, db_abs * np.abs(wp)
        db = sig * (dxn - xn * (dxn * xn).mean(1, keepdims=True))
        db_abs = sig * (dxn_abs + np.abs(xn) * (dxn_abs * np.abs(xn)).mean(1, keepdims=True))
    out["d_x"] = (db, db_abs)
    return out
