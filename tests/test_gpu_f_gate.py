"""The gate, the balance loss and their gradient against the float64 oracle.

Choices and counts are exact. Floating results carry float32 rounding:
tolerances are counted in half steps of float32 (2^-24) per operation, and a
BF16 gradient adds half a BF16 step (2^-8).
"""
import numpy as np
import pytest
import torch

import oracle.gate as G
from _block_cases import DEV, EPS32, HALF_BF16, as_stored, gate_logits, grad_bound, guarded, to_dev, torch_dtype

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import nvfp4_quantized_moe_amd as nv
    return nv


def case(T, E, k, score=G.SOFTMAX, dtype="f32", kind="plain", **kw):
    d = dict(T=T, E=E, k=k, score=score, dtype=dtype, kind=kind, bias=False, groups=1, top=1, renorm=True, mask=False)
    d.update(kw)
    return d


CASES = [
    case(1, 1, 1), case(1, 384, 8), case(3, 7, 7, G.SIGMOID), case(70, 60, 4, dtype="bf16", mask=True),
    case(65, 384, 8, kind="ties", dtype="bf16"), case(33, 256, 8, G.SIGMOID, kind="ties", bias=True, groups=8, top=4),
    case(40, 256, 8, G.SIGMOID, dtype="bf16", kind="ties", groups=8, top=3),
    case(41, 384, 6, G.SIGMOID, bias=True, groups=8, top=4, mask=True),
    case(37, 384, 8, G.SQRT_SOFTPLUS, dtype="bf16", bias=True), case(29, 383, 9, G.SOFTMAX, bias=True, groups=1),
    case(31, 96, 5, G.SOFTMAX, kind="ties", groups=32, top=7), case(30, 512, 12, G.SQRT_SOFTPLUS, kind="wide"),
    case(32, 128, 8, G.SOFTMAX, kind="wide", bias=True, groups=4, top=2, renorm=False),
    case(26, 64, 8, G.SOFTMAX, kind="holes"), case(26, 64, 8, G.SIGMOID, kind="holes", bias=True, groups=8, top=4),
    case(27, 200, 16, G.SQRT_SOFTPLUS, kind="holes", dtype="bf16", renorm=False),
    case(25, 1024, 64, G.SIGMOID, renorm=False), case(21, 1000, 63, G.SOFTMAX, bias=True, renorm=False),
    case(24, 100, 64, G.SOFTMAX, dtype="bf16"), case(2050, 48, 2, G.SIGMOID, mask=True),
    case(64, 64, 4, G.SIGMOID, groups=64, top=10), case(22, 24, 20, G.SIGMOID, kind="holes", groups=2, top=2),
]
IDS = [f"{i}-T{c['T']}-E{c['E']}-k{c['k']}-s{c['score']}-{c['kind']}" for i, c in enumerate(CASES)]


def setup(c, seed):
    x = gate_logits(c, seed)
    rng = np.random.default_rng(seed + 1000)
    bias = np.round(rng.standard_normal(c["E"]) * 0.1, 2).astype(np.float32) if c["bias"] else None
    mask = (rng.random(c["T"]) > 0.2).astype(np.uint8) if c["mask"] else None
    dev = to_dev(x.astype(np.float32), torch_dtype(c["dtype"]))
    if mask is not None:
        dev[torch.from_numpy(mask).to(DEV) == 0] = float("nan")  # padding may hold anything
    return x, bias, mask, dev


def gate(nv, c, dev, bias, mask, **kw):
    return nv.moe_gate_topk(dev, c["k"], score=c["score"], bias=None if bias is None else to_dev(bias),
                            token_mask=None if mask is None else to_dev(mask), n_group=c["groups"],
                            topk_group=c["top"], renormalize=c["renorm"], scale=2.5, **kw)


@pytest.mark.parametrize("c", CASES, ids=IDS)
def test_choices_and_weights(nv, c):
    x, bias, mask, dev = setup(c, 7)
    T, E, k = c["T"], c["E"], c["k"]
    ids, ids_ok = guarded((T, k), torch.int32, -77)
    w, w_ok = guarded((T, k), torch.float32, -77.0)
    gate(nv, c, dev, bias, mask, topk_ids=ids, topk_w=w)
    assert ids_ok() and w_ok()
    ref_ids, ref_w = G.gate_topk(x, k, c["score"], bias, mask, c["groups"], c["top"], c["renorm"], 2.5)
    assert np.array_equal(ids.cpu().numpy(), ref_ids)
    got = w.cpu().numpy().astype(np.float64)
    # exp and log within 2 steps, at most k additions and 6 other roundings, the argument x - max of a softmax
    # |x - max| half steps; float32 results below 2^-126 may be lost
    fin = np.where(np.isfinite(x), x, 0.0)
    span = np.minimum(200.0, np.abs(fin).max(1, keepdims=True) * 2) if c["score"] == G.SOFTMAX else 0.0
    tol = (16 + k + span) * EPS32 * ref_w + 2.5 * 2.0 ** -126
    assert (np.abs(got - ref_w) <= tol).all(), float(np.max(np.abs(got - ref_w) / np.maximum(ref_w, 1e-30)))


@pytest.mark.parametrize("E,k,score,groups,top", [
    (384, 8, G.SIGMOID, 1, 1), (40, 8, G.SIGMOID, 1, 1), (384, 20, G.SIGMOID, 1, 1), (1000, 16, G.SQRT_SOFTPLUS, 1, 1),
    (63, 5, G.SQRT_SOFTPLUS, 1, 1), (256, 8, G.SIGMOID, 8, 4), (96, 5, G.SOFTMAX, 32, 7), (64, 4, G.SOFTMAX, 1, 1),
    (512, 16, G.SOFTMAX, 4, 2), (300, 64, G.SIGMOID, 1, 1)])
def test_crowded_keys(nv, E, k, score, groups, top):
    """Rows whose keys lie closer together than float32 can tell apart: all of them, or a crowd around the k-th. The
    logits differ by steps of 2^-24, the biases by about as much; float64 separates them by far more than its own
    rounding."""
    T = 34
    rng = np.random.default_rng(E + k)
    x = (0.5 + rng.integers(0, 400, (T, E)) * 2.0 ** -24)
    x[::2] += np.where(rng.random((T // 2, E)) < 0.5, 0.0, -1.0)                 # half of the row out of question
    x[::4, : k // 2] += 1.0                                                       # the first choices clear
    x[1::4, ::3] = -np.inf
    x = as_stored(x, "f32")
    bias = (rng.standard_normal(E) * 1e-7).astype(np.float32)
    ref_ids, _ = G.gate_topk(x, k, score, bias, None, groups, top, True, 1.0)
    ids, _ = nv.moe_gate_topk(to_dev(x.astype(np.float32)), k, score=score, bias=to_dev(bias), n_group=groups,
                              topk_group=top)
    assert np.array_equal(ids.cpu().numpy(), ref_ids)


def seq_of(T, cu):
    seq = np.full(T, -1)
    for b, (lo, hi) in enumerate(G.spans(T, cu)):
        seq[lo:hi] = b
    return seq


def sequences(T, kind):
    if kind is None:
        return None
    if kind == "gaps":     # empty ones in front, between and behind; tokens before the first and after the last
        lo, hi = T // 8, T - T // 8
        return np.array([lo, lo, (lo + hi) // 2, (lo + hi) // 2, hi, hi], np.int32)
    return np.sort(np.concatenate([[0, T], np.random.default_rng(3).integers(0, T + 1, kind - 1)])).astype(np.int32)


@pytest.mark.parametrize("seqs", [None, "gaps", 70], ids=["one", "gaps", "seventy"])
@pytest.mark.parametrize("c", [c for c in CASES if c["k"] <= 20 and c["groups"] in (1, 8)],
                         ids=[i for i, c in zip(IDS, CASES) if c["k"] <= 20 and c["groups"] in (1, 8)])
def test_balance_loss_and_gradient(nv, c, seqs):
    x, bias, mask, dev = setup(c, 11)
    T, E, k = c["T"], c["E"], c["k"]
    cu = sequences(T, seqs)
    rng = np.random.default_rng(5)
    ids, _ = G.gate_topk(x, k, c["score"], bias, mask, c["groups"], c["top"])
    if T > 8:
        ids[6, 0] = E + 5            # another rank's
        ids[7, -1] = ids[7, 0]       # listed twice
    d_ids = to_dev(ids)
    d_cu = None if cu is None else to_dev(cu)
    d_mask = None if mask is None else to_dev(mask)
    loss, counts, tokens = nv.moe_balance_loss(dev, d_ids, score=c["score"], token_mask=d_mask, cu_seqlens=d_cu)
    ref_loss, ref_counts, ref_tokens = G.balance_loss(x, ids, c["score"], mask, cu)
    assert np.array_equal(counts.cpu().numpy(), ref_counts)
    assert np.array_equal(tokens.cpu().numpy(), ref_tokens)
    # every q carries at most (16 + E/64 + 6 + span) half steps, the sums over tokens are of positive terms with at
    # most 64 float32 additions in a row; logsumexp adds its own 4 roundings at the size of the largest |x|
    fin = x[np.isfinite(x) & (np.abs(x) < 1e30)]
    span = 2 * np.abs(fin).max() if len(fin) else 0.0
    got = loss.cpu().numpy().astype(np.float64)
    assert abs(got[0] - ref_loss[0]) <= (110 + span) * EPS32 * ref_loss[0]
    if ref_loss[1] < 1e30:  # rows of the type's lowest value alone have a squared log-sum past float32
        assert abs(got[1] - ref_loss[1]) <= 16 * EPS32 * (np.sqrt(ref_loss[1]) + span + 1) ** 2
    d_w = rng.standard_normal((T, k)).astype(np.float32)
    d_loss = np.array([0.9, 0.02], np.float32)
    seq = seq_of(T, cu)
    live = G.live_tokens(x, mask)
    for use_w, use_loss in ((True, False), (False, True), (True, True)):
        out, intact = guarded((T, E), torch_dtype(c["dtype"]), 7.0)
        nv.moe_gate_backward(dev, d_ids, score=c["score"], renormalize=c["renorm"], scale=1.5, token_mask=d_mask,
                             d_topk_w=to_dev(d_w) if use_w else None, d_loss=to_dev(d_loss) if use_loss else None,
                             counts=counts, tokens=tokens, cu_seqlens=d_cu, d_logits=out)
        assert intact()
        args = dict(d_w=d_w if use_w else None, d_loss=d_loss if use_loss else None)
        ref = G.gate_backward(x, ids, c["score"], c["renorm"], 1.5, mask, counts=ref_counts, tokens=ref_tokens, cu=cu,
                              **args)
        got = out.float().cpu().numpy().astype(np.float64)
        assert not got[~live].any()
        tol = grad_bound(x, ids, 1.5 * d_w if use_w else None, c["score"], c["renorm"], mask, args["d_loss"],
                         ref_counts, ref_tokens, seq) + 2.0 ** -120
        if c["dtype"] == "bf16":
            tol = tol * (1 + HALF_BF16) + HALF_BF16 * np.abs(ref)
        fine = np.abs(got - ref) <= tol
        low = np.abs(np.where(np.isfinite(x), x, 0.0)).max(1) > 1e30   # see above: compared where lse is ordinary
        low &= x.max(1) < -1e30
        assert fine[~low].all(), (use_w, use_loss, float(np.max(np.abs(got - ref)[~low] / tol[~low])))


def test_empty_batch(nv):
    x = torch.empty((0, 16), device=DEV)
    ids, w = nv.moe_gate_topk(x, 2)
    assert ids.shape == (0, 2) and w.shape == (0, 2)
    loss, counts, tokens = nv.moe_balance_loss(x, ids, cu_seqlens=torch.zeros(4, dtype=torch.int32, device=DEV))
    assert not loss.any() and not counts.any() and tokens.tolist() == [0] * 5
    assert nv.moe_gate_backward(x, ids, d_topk_w=w).shape == (0, 16)


def test_equal_on_every_run_and_in_a_graph(nv):
    """Bit for bit: two eager runs, a side stream, and replays of one captured graph with eager work between them."""
    c = case(515, 384, 8, G.SIGMOID, bias=True, groups=8, top=4, mask=True)
    x, bias, mask, dev = setup(c, 3)
    dev = torch.nan_to_num(dev)
    cu = to_dev(sequences(515, 5))
    d_bias, d_mask = to_dev(bias), to_dev(mask)
    d_w = torch.randn(515, 8, device=DEV)
    d_loss = torch.tensor([0.5, 0.1], device=DEV)
    ws = torch.empty(nv.moe_balance_loss_ws_bytes(515, 384, 5), dtype=torch.uint8, device=DEV)
    bufs = dict(ids=torch.empty(515, 8, dtype=torch.int32, device=DEV), w=torch.empty(515, 8, device=DEV),
                loss=torch.empty(2, device=DEV), counts=torch.empty(5, 384, dtype=torch.int32, device=DEV),
                tokens=torch.empty(7, dtype=torch.int32, device=DEV), d=torch.empty(515, 384, device=DEV))

    def step():
        nv.moe_gate_topk(dev, 8, G.SIGMOID, d_bias, d_mask, 8, 4, True, 2.5, bufs["ids"], bufs["w"])
        nv.moe_balance_loss(dev, bufs["ids"], G.SIGMOID, d_mask, cu, bufs["loss"], bufs["counts"], bufs["tokens"], ws)
        nv.moe_gate_backward(dev, bufs["ids"], G.SIGMOID, True, 2.5, d_mask, d_w, d_loss, bufs["counts"],
                             bufs["tokens"], cu, bufs["d"])

    def snap():
        torch.cuda.synchronize()
        return {n: b.clone() for n, b in bufs.items()}

    def wipe():
        for b in bufs.values():
            b.fill_(-3)
        ws.fill_(0xA5)

    step()
    first = snap()
    wipe()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    second = snap()
    assert all(torch.equal(first[n], second[n]) for n in bufs)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(4):
        wipe()
        g.replay()
        again = snap()
        assert all(torch.equal(first[n], again[n]) for n in bufs)


def test_choices_feed_the_route(nv):
    c = case(300, 64, 6, G.SIGMOID, kind="holes", bias=True, groups=8, top=4, mask=True)
    x, bias, mask, dev = setup(c, 5)
    ids, w = gate(nv, c, dev, bias, mask)
    r = nv.moe_route_slots(ids, w, 16, 24, 32)
    _, counts, _ = nv.moe_balance_loss(dev, ids, score=c["score"], token_mask=to_dev(mask))
    assert torch.equal(r["counts"], counts[0, 16:40])
    assert int(r["offsets"][-1]) == int(counts[0, 16:40].sum())
