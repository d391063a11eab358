"""The gate oracle: worked examples, and its gradients against differences (CPU)."""
import numpy as np
import pytest

import oracle.gate as G


def test_worked_choices():
    x = np.array([[0.0, 2.0, 2.0, -1.0], [-np.inf, -np.inf, 3.0, -np.inf], [-np.inf] * 4, [1.0, 1.0, 1.0, 1.0]])
    ids, w = G.gate_topk(x, 2, G.SOFTMAX, scale=2.0)
    assert ids.tolist() == [[1, 2], [2, -1], [-1, -1], [0, 1]]
    assert np.allclose(w, [[1, 1], [2, 0], [0, 0], [1, 1]])
    # a bias moves the choice and not the weight
    ids, w = G.gate_topk(x[:1], 1, G.SIGMOID, bias=np.array([0.0, 0, 0, 5]), renormalize=False)
    assert ids[0, 0] == 3 and np.isclose(w[0, 0], 1 / (1 + np.e))
    # groups {0, 1} and {2, 3}: the pair (1.0, 0.9) beats a lone 1.5 beside -3
    g = np.array([[1.0, 0.9, 1.5, -3.0]])
    ids, _ = G.gate_topk(g, 2, G.SIGMOID, n_group=2, topk_group=1)
    assert ids.tolist() == [[0, 1]]
    # a masked token
    ids, w = G.gate_topk(x[:1], 2, G.SOFTMAX, mask=np.array([0]))
    assert ids.tolist() == [[-1, -1]] and not w.any()


def test_uniform_routing_has_balance_loss_one():
    # every expert equally likely and equally often chosen
    E, k = 8, 2
    x = np.zeros((E, E))
    ids = np.array([[t, (t + 1) % E] for t in range(E)], np.int32)
    loss, counts, tokens = G.balance_loss(x, ids, G.SOFTMAX)
    assert np.allclose(loss, [1.0, np.log(E) ** 2]) and (counts == 2).all() and tokens.tolist() == [8, 8, 1]
    # all tokens on one expert: E
    x[:, 0] = 60.0
    loss, _, _ = G.balance_loss(x, np.zeros((E, 1), np.int32), G.SOFTMAX)
    assert np.isclose(loss[0], E)


@pytest.mark.parametrize("score", [G.SOFTMAX, G.SIGMOID, G.SQRT_SOFTPLUS])
@pytest.mark.parametrize("renormalize", [True, False])
def test_gradients_equal_differences(score, renormalize):
    rng = np.random.default_rng(score * 2 + renormalize)
    T, E, k = 9, 7, 3
    x = rng.standard_normal((T, E)) * 2
    ids, _ = G.gate_topk(x, k, score)
    ids[4, 1] = ids[4, 0]      # an expert listed twice
    ids[5, 2] = -1
    mask = np.ones(T, np.uint8)
    mask[3] = 0
    cu = np.array([0, 4, 4, 8])  # an empty sequence, and a token behind the last
    d_w, d_loss = rng.standard_normal((T, k)), np.array([0.7, 0.3])
    _, counts, tokens = G.balance_loss(x, ids, score, mask, cu)
    got = G.gate_backward(x, ids, score, renormalize, 1.5, mask, d_w, d_loss, counts, tokens, cu)

    def value(z):
        loss, _, _ = G.balance_loss(z, ids, score, mask, cu)
        w = np.stack([G.weights(z[t], ids[t], score, renormalize, 1.5) * mask[t] for t in range(T)])
        return (w * d_w).sum() + (loss * d_loss).sum()

    h = 1e-5
    for t in range(T):
        for e in range(E):
            up, down = x.copy(), x.copy()
            up[t, e] += h
            down[t, e] -= h
            # central differences: error h^2 times the third derivative (of order 10 here) + rounding 1e-16 / h
            assert abs((value(up) - value(down)) / (2 * h) - got[t, e]) < 1e-8
    assert not got[3].any()
