"""The layer norm's oracle: worked rows, and its gradients against differences (CPU)."""
import numpy as np

import oracle.layer_norm as LN


def test_worked_rows():
    r = np.array([[1.0, 3.0, 5.0, 7.0], [2.0, 2.0, 2.0, 2.0]])
    y = LN.forward(r, np.array([1.0, 2.0, 1.0, 1.0]), np.array([0.0, 0.0, 10.0, 0.0]), eps=0.0 + 4.0)
    assert np.allclose(y, [[-1.0, -2.0 / 3, 10 + 1.0 / 3, 1.0], [0, 0, 10, 0]])     # var 5, sqrt(5 + 4) = 3
    shifted = LN.forward(r + 1000.0)
    assert np.allclose(shifted, LN.forward(r), atol=1e-9)
    assert LN.update(np.ones((1, 2)), np.full((1, 2), 3.0), 0.5)[0].tolist() == [[3.5, 3.5]]


def test_gradients_against_differences():
    rng = np.random.default_rng(0)
    T, H, eps, scale = 3, 7, 1e-3, 0.75
    x, res, dy, dro = (rng.standard_normal((T, H)) for _ in range(4))
    w, b = 1 + 0.3 * rng.standard_normal(H), rng.standard_normal(H)

    def loss(x, res, w, b):
        r = LN.update(x, res, scale)[0]
        return (LN.forward(r, w, b, eps) * dy).sum() + (r * dro).sum()
    got = LN.backward(dy, dro, LN.update(x, res, scale)[0], w, scale, eps)
    for i, name in enumerate(("d_x", "d_residual", "d_w", "d_b")):
        args = [x, res, w, b]
        want = np.zeros_like(args[i])
        for at in np.ndindex(*want.shape):
            h = 1e-6
            for sign in (1, -1):
                v = [a.copy() for a in args]
                v[i][at] += sign * h
                want[at] += sign * loss(*v) / (2 * h)
        assert np.allclose(got[name][0], want, rtol=1e-6, atol=1e-7), name
        assert (np.abs(got[name][0]) <= got[name][1] + 1e-12).all()
