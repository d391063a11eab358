"""The norm oracle's gradients against differences (CPU)."""
import numpy as np
import pytest

import oracle.norm as N


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [None, "channel", "token"])
def test_gradients_equal_differences(post, gate):
    rng = np.random.default_rng(3)
    T, H = 3, 8
    p = dict(x=rng.standard_normal((T, H)), residual=rng.standard_normal((T, H)), w_pre=rng.standard_normal(H) + 1)
    if post:
        p["w_post"] = rng.standard_normal(H)
    if gate:
        p["gate"] = rng.standard_normal(H if gate == "channel" else (T, 1))
    d_y, d_res = rng.standard_normal((T, H)), rng.standard_normal((T, H))

    def value(**q):
        r, _ = N.update(q["x"], q["residual"], q.get("w_post"), q.get("gate"), 0.7, 1e-3)
        return (N.normalize(r, q["w_pre"], 1e-3) * d_y).sum() + (r * d_res).sum()

    r, _ = N.update(p["x"], p["residual"], p.get("w_post"), p.get("gate"), 0.7, 1e-3)
    got = N.backward(d_y, d_res, p["x"], r, p["w_pre"], p.get("w_post"), p.get("gate"), 0.7, 1e-3)
    for name, arr in p.items():
        d = got["d_" + name][0]
        assert d.shape == arr.shape
        for i in np.ndindex(arr.shape):
            up, down = arr.copy(), arr.copy()
            up[i] += 1e-5
            down[i] -= 1e-5
            diff = (value(**{**p, name: up}) - value(**{**p, name: down})) / 2e-5
            # h^2 = 1e-10 times a third derivative of order 10, rounding 1e-15 / h
            assert abs(diff - d[i]) < 2e-8 * max(1.0, abs(d[i])), (name, i)


def test_rms_of_the_result_is_one():
    x = np.random.default_rng(0).standard_normal((4, 64)) * 5
    y = N.normalize(x, np.ones(64), 0.0)
    assert np.allclose((y * y).mean(1), 1.0)
