"""The gate, the balance loss and their gradient where float32 keys, sums or scores run out: against the float64
oracle, with the tolerances of test_gpu_f_gate.py."""
import numpy as np
import pytest
import torch

import oracle.gate as G
from _block_cases import DEV, EPS32, HALF_BF16, as_stored, grad_bound, to_dev, torch_dtype

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import nvfp4_quantized_moe_amd as nv
    return nv


def choices(nv, x, k, score, bias=None, groups=1, top=1, dtype="f32"):
    """ids of the kernel and of the oracle."""
    ids, _ = nv.moe_gate_topk(to_dev(x.astype(np.float32), torch_dtype(dtype)), k, score=score,
                              bias=None if bias is None else to_dev(bias), n_group=groups, topk_group=top)
    return ids.cpu().numpy(), G.gate_topk(x, k, score, bias, None, groups, top)[0]


def wrong_rows(got, ref):
    return int((got != ref).any(1).sum())


@pytest.mark.parametrize("k", [2, 7, 20])
def test_a_bias_that_cancels_its_score(nv, k):
    """k - 1 clear choices, then scores of 2e-8 and 1e-8 without a bias, and further down an expert whose bias is the
    negative of its rounded score: what is left of its key is the rounding, often more than 2e-8."""
    E, low = 64, 32
    rng = np.random.default_rng(k)
    for _ in range(10):
        bias = np.zeros(E, np.float32)
        at = rng.uniform(1.5, 3.0, E).astype(np.float32)
        bias[low + 2:] = -(1.0 / (1.0 + np.exp(-at[low + 2:].astype(np.float64)))).astype(np.float32)
        x = np.full((E - low - 2, E), -np.inf)
        x[:, :k - 1] = rng.uniform(2.0, 6.0, (len(x), k - 1))
        x[:, low - 1] = np.log(2e-8)
        x[:, low] = np.log(1e-8)
        for t in range(len(x)):
            x[t, low + 2 + t] = at[low + 2 + t]
        got, ref = choices(nv, as_stored(x, "f32"), k, G.SIGMOID, bias)
        assert wrong_rows(got, ref) == 0


@pytest.mark.parametrize("score,k,row,expected", [
    (G.SIGMOID, 1, [20, 20, 21, 0, 0, 0, 0, 0], [2]),                # 1 in float32, all three of the highest
    (G.SIGMOID, 2, [20, 19, 20, 21, 0, 0, 0, 0], [3, 0]),
    (G.SOFTMAX, 2, [200, 1, 1, 2, 0, 0, 0, 0], [0, 3]),              # 0 in float32, all but the first
    (G.SQRT_SOFTPLUS, 1, [-200, -200, -190, -300, -300, -300, -300, -300], [2]),
])
def test_copies_at_the_last_choice(nv, score, k, row, expected):
    """The k-th and the next key are copies of one logit, and float32 cannot tell a higher one from them."""
    x, bias = np.array([row], np.float64), np.zeros(len(row), np.float32)
    got, ref = choices(nv, x, k, score, bias)
    assert got.tolist() == ref.tolist() == [expected]


@pytest.mark.parametrize("k", [1, 2, 6, 20])
@pytest.mark.parametrize("E,score,scale,groups,top,biased", [
    (256, G.SIGMOID, 8, 1, 1, True), (256, G.SIGMOID, 8, 8, 4, False), (384, G.SIGMOID, 12, 8, 3, False),
    (60, G.SOFTMAX, 40, 1, 1, True), (256, G.SOFTMAX, 40, 8, 4, False), (96, G.SQRT_SOFTPLUS, 60, 4, 2, False),
    (300, G.SQRT_SOFTPLUS, 60, 1, 1, True)])
def test_saturated_rows_of_few_values(nv, E, score, scale, groups, top, biased, k):
    """BF16 logits of a wide range: many equal ones, many whose scores float32 rounds to the same, and no bias (or
    one of zeros) to tell them apart."""
    rng = np.random.default_rng(E + k)
    x = as_stored(rng.standard_normal((400, E)) * scale, "bf16")
    x[::4] = np.round(x[::4])
    got, ref = choices(nv, x, k, score, np.zeros(E, np.float32) if biased else None, groups, top, "bf16")
    assert wrong_rows(got, ref) == 0


@pytest.mark.parametrize("offset", [0.0, 1000.0, -30000.0])
def test_softmax_gradient_of_shifted_rows(nv, offset):
    """Softmax does not see a common offset of a row's logits; neither does the gradient through weights that are not
    renormalized. (Logits in steps of 2^-8, so that float32 holds them with the offset.)"""
    T, E, k = 200, 90, 6
    rng = np.random.default_rng(4)
    x = np.round(rng.standard_normal((T, E)) * 1.5 * 256) / 256 + offset
    assert np.array_equal(as_stored(x, "f32"), x)
    ids, _ = G.gate_topk(x, k, G.SOFTMAX)
    d_w = rng.standard_normal((T, k)).astype(np.float32)
    got = nv.moe_gate_backward(to_dev(x.astype(np.float32)), to_dev(ids), G.SOFTMAX, False, 1.5, d_topk_w=to_dev(d_w))
    ref = G.gate_backward(x, ids, G.SOFTMAX, False, 1.5, d_w=d_w)
    tol = grad_bound(x, ids, 1.5 * d_w, G.SOFTMAX, False, None, None, None, None, np.full(T, -1)) + 2.0 ** -120
    worst = float(np.max(np.abs(got.double().cpu().numpy() - ref) / tol))
    assert worst <= 1


@pytest.mark.parametrize("score", [G.SOFTMAX, G.SIGMOID, G.SQRT_SOFTPLUS])
@pytest.mark.parametrize("k", [1, 4])
def test_a_single_renormalized_choice_has_no_gradient(nv, k, score):
    """Its weight is the scale whatever its logit: k = 1, or one expert that the token may use."""
    T, E = 300, 40
    rng = np.random.default_rng(k)
    x = as_stored(rng.standard_normal((T, E)) * 3, "f32")
    if k > 1:
        keep = x[np.arange(T), np.arange(T) % E]
        x[:] = -np.inf
        x[np.arange(T), np.arange(T) % E] = keep
    ids, w = nv.moe_gate_topk(to_dev(x.astype(np.float32)), k, score, scale=2.5)
    assert (ids[:, 1:] == -1).all()
    d_w = to_dev(rng.standard_normal((T, k)).astype(np.float32))
    d = nv.moe_gate_backward(to_dev(x.astype(np.float32)), ids, score, True, 2.5, d_topk_w=d_w)
    assert not d.any()


@pytest.mark.parametrize("score", [G.SIGMOID, G.SQRT_SOFTPLUS])
@pytest.mark.parametrize("level", [-15.0, -25.0, -88.0, -110.0, -180.0, -400.0])
def test_rows_far_below_zero(nv, level, score):
    """Scores that are divided by their sum depend on their ratios alone, also where float32 cannot hold them."""
    T, E, k = 90, 70, 5
    rng = np.random.default_rng(int(-level))
    x = as_stored(level + rng.standard_normal((T, E)) * 4, "f32")
    x[::3, 7:] = -np.inf
    dev = to_dev(x.astype(np.float32))
    bias = rng.standard_normal(E).astype(np.float32)   # float64 keys of such scores would be those of the bias
    ids, w = nv.moe_gate_topk(dev, k, score, bias=to_dev(bias), scale=2.5)
    ref_ids, ref_w = G.gate_topk(x, k, score, bias, scale=2.5)
    assert wrong_rows(ids.cpu().numpy(), ref_ids) == 0
    # exp within 2 steps, k additions and 6 other roundings, and |x - max| half steps of an exponential's argument;
    # beside a sum of at least 2^-28 scores under 2^-126 may be lost
    fin = np.where(x > -np.inf, x, np.nan)
    span = np.nanmax(fin, 1) - np.nanmin(fin, 1)
    tol = (16 + k + 2 * span[:, None]) * EPS32 * ref_w + 2.5 * 2.0 ** -98
    assert float(np.max(np.abs(w.double().cpu().numpy() - ref_w) / tol)) <= 1
    d_w, d_loss = rng.standard_normal((T, k)).astype(np.float32), np.array([0.9, 0.0], np.float32)
    loss, counts, tokens = nv.moe_balance_loss(dev, ids, score)
    ref_loss, ref_counts, ref_tokens = G.balance_loss(x, ref_ids, score)
    assert abs(float(loss[0]) - ref_loss[0]) <= (110 + 2 * span.max()) * EPS32 * ref_loss[0]
    for use_w, use_loss in ((True, False), (False, True)):
        got = nv.moe_gate_backward(dev, ids, score, True, 1.5, d_topk_w=to_dev(d_w) if use_w else None,
                                   d_loss=to_dev(d_loss) if use_loss else None, counts=counts, tokens=tokens)
        args = dict(d_w=d_w if use_w else None, d_loss=d_loss if use_loss else None)
        ref = G.gate_backward(x, ref_ids, score, True, 1.5, counts=ref_counts, tokens=ref_tokens, **args)
        tol = grad_bound(x, ref_ids, 1.5 * d_w if use_w else None, score, True, None, args["d_loss"], ref_counts,
                         ref_tokens, np.zeros(T, int)) + 2.0 ** -98
        assert float(np.max(np.abs(got.double().cpu().numpy() - ref) / tol)) <= 1, (use_w, use_loss)


@pytest.mark.parametrize("score,row", [(G.SIGMOID, [1.1, 0.0]), (G.SIGMOID, [-1.3, 0.4]), (G.SOFTMAX, [0.7, 0.1]),
                                       (G.SQRT_SOFTPLUS, [2.0, -0.5])])
def test_sums_over_very_many_tokens(nv, score, row):
    """Equal rows, so that additions that are rounded all round the same way: 2^25 tokens give a wave 8192 of them."""
    T, E = (1 << 25) + 77, 2
    x = as_stored(np.array([row]), "f32")
    dev = to_dev(x.astype(np.float32)).expand(T, E).contiguous()
    ids = torch.zeros((T, 1), dtype=torch.int32, device=DEV)
    loss, counts, tokens = nv.moe_balance_loss(dev, ids, score)
    assert counts.tolist() == [[T, 0]] and tokens.tolist() == [T, T, 1]
    s = G.scores(x, score)[0]
    ref = E * s[0] / s.sum()
    # as in test_balance_loss_and_gradient: a share within its own roundings, at most 64 float32 additions in a row
    assert abs(float(loss[0]) - ref) <= (110 + 2 * np.abs(x).max()) * EPS32 * ref
    lse = np.log(np.exp(x).sum())
    assert abs(float(loss[1]) - lse ** 2) <= 16 * EPS32 * (abs(lse) + 2 * np.abs(x).max() + 1) ** 2


@pytest.mark.parametrize("cu", [None, [0, 11000, 11000, 11003, 11100, 11900, 12010]], ids=["one", "one-long"])
@pytest.mark.parametrize("T,E,k,score,dtype", [(12011, 24, 3, G.SIGMOID, "f32"), (33000, 10, 2, G.SOFTMAX, "bf16"),
                                               (20000, 70, 1, G.SQRT_SOFTPLUS, "f32")])
def test_balance_loss_of_large_batches(nv, T, E, k, score, dtype, cu):
    """More than eight tokens to a partial sum; a long sequence beside short ones."""
    rng = np.random.default_rng(T)
    x = as_stored(rng.standard_normal((T, E)) * 1.5 + rng.standard_normal(E), dtype)
    ids = np.argsort(-x, 1, kind="stable")[:, :k].astype(np.int32)
    mask = (rng.random(T) > 0.1).astype(np.uint8)
    cu = None if cu is None else np.array(cu, np.int32)
    dev = to_dev(x.astype(np.float32), torch_dtype(dtype))
    loss, counts, tokens = nv.moe_balance_loss(dev, to_dev(ids), score, to_dev(mask), None if cu is None else to_dev(cu))
    ref_loss, ref_counts, ref_tokens = G.balance_loss(x, ids, score, mask, cu)
    assert np.array_equal(counts.cpu().numpy(), ref_counts) and np.array_equal(tokens.cpu().numpy(), ref_tokens)
    span = 2 * np.abs(x).max()
    got = loss.double().cpu().numpy()
    assert abs(got[0] - ref_loss[0]) <= (110 + span) * EPS32 * ref_loss[0]
    assert abs(got[1] - ref_loss[1]) <= 16 * EPS32 * (np.sqrt(ref_loss[1]) + span + 1) ** 2
    d_loss = np.array([0.9, 0.02], np.float32)
    d = nv.moe_gate_backward(dev, to_dev(ids), score, token_mask=to_dev(mask), d_loss=to_dev(d_loss), counts=counts,
                             tokens=tokens, cu_seqlens=None if cu is None else to_dev(cu))
    ref = G.gate_backward(x, ids, score, mask=mask, d_loss=d_loss, counts=ref_counts, tokens=ref_tokens, cu=cu)
    seq = np.full(T, -1)
    for b, (lo, hi) in enumerate(G.spans(T, cu)):
        seq[lo:hi] = b
    tol = grad_bound(x, ids, None, score, True, mask, d_loss, ref_counts, ref_tokens, seq) + 2.0 ** -120
    if dtype == "bf16":
        tol = tol * (1 + HALF_BF16) + HALF_BF16 * np.abs(ref)
    assert (np.abs(d.double().cpu().numpy() - ref) <= tol).all()


@pytest.mark.parametrize("score,level,bias_size", [(G.SIGMOID, -87.35, 0.0), (G.SQRT_SOFTPLUS, -174.7, 0.0),
                                                   (G.SOFTMAX, -87.35, 0.0), (G.SIGMOID, -87.35, 1e-38)])
def test_scores_at_the_end_of_float32(nv, score, level, bias_size):
    """Scores about 2^-126: a sum (of a group's two highest, or with a bias) of what float32 keeps of one and loses of
    another does not have the order of the sums."""
    T, E = 600, 64
    rng = np.random.default_rng(9)
    x = level + rng.uniform(-0.15, 0.15, (T, E))
    if score == G.SOFTMAX:
        x[:, 0] = 0.0
    x = as_stored(x, "f32")
    bias = (rng.uniform(-1, 1, E) * bias_size).astype(np.float32) if bias_size else None
    for groups, top in ((1, 1), (16, 5)) if bias_size else ((16, 5), (32, 3)):
        got, ref = choices(nv, x, 3, score, bias, groups, top)
        assert wrong_rows(got, ref) == 0, groups


@pytest.mark.parametrize("score,level", [(G.SIGMOID, -500.0), (G.SIGMOID, -712.0), (G.SIGMOID, -722.0),
                                         (G.SQRT_SOFTPLUS, -650.0), (G.SOFTMAX, -722.0)])
@pytest.mark.parametrize("groups,top", [(1, 1), (4, 2)])
def test_keys_of_float64_down_to_its_end(nv, score, level, groups, top):
    """Scores that float64 still tells apart (steps of 1/4 of the logit, its last digits above 2^-1074)."""
    T, E = 300, 40
    rng = np.random.default_rng(int(-level))
    x = level + rng.integers(-20, 21, (T, E)) / 4.0
    if score == G.SOFTMAX:
        x[:, ::10] = 0.0
    got, ref = choices(nv, x, 7, score, np.zeros(E, np.float32), groups, top)
    assert wrong_rows(got, ref) == 0
