"""The expert layer for a few tokens against float64, step by step: h, which the workspace keeps, from the inputs, and
the output from that h. A weight times an activation is exact in float32 (6 and 8 significant bits); a sum of K of them
has at most K / 16 + 16 + 8 roundings behind any term (the instructions of a wave one after the other, 16 products of
each in any order, the waves), each within one float32 step of the terms' sum, and the output one more per expert.
"""
import numpy as np
import pytest
import torch

import oracle as O
import oracle.few as F
from _block_cases import DEV, EPS32, HALF_BF16, guarded, to_dev

pytestmark = pytest.mark.gpu
STEP = 2 * EPS32


@pytest.fixture(scope="module")
def nv():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import nvfp4_quantized_moe_amd as nv
    return nv


def matrices(g, L, N, K):
    """NVFP4 of L matrices with every code and scales of all sizes."""
    q = torch.randint(0, 256, (L, N, K // 2), dtype=torch.uint8, device=DEV, generator=g)
    sf = torch.randint(0x28, 0x48, (L, N, K // 16), dtype=torch.uint8, device=DEV, generator=g)
    sf[:, 0, 0], sf[:, N - 1, -1] = 0x7E, 0x01   # the largest and the smallest scale
    return q, sf


def values(q, sf):
    """float64 of a matrix, without its global scale."""
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device=DEV)
    v = torch.stack([table[(q & 15).long()], table[(q >> 4).long()]], -1).reshape(q.shape[0], -1)
    return v * sf.view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)


def layer(nv, L, H, I, dual, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    w1, w2 = matrices(g, L, 2 * I, H), matrices(g, L, H, I)
    gs1 = (0.5 + torch.rand((L, 2) if dual else (L,), device=DEV, generator=g)) * 0.5 * H ** -0.5
    gs2 = (0.5 + torch.rand(L, device=DEV, generator=g)) * I ** -0.5
    return nv.MoEWeights(nv.nvfp4_pack_weights(*w1), gs1, nv.nvfp4_pack_weights(*w2), gs2), w1, w2, g


def choices(kind, T, k, E, start, L, seed):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    if kind == "masked":
        ids[rng.random(T) < 0.4] = -1
        ids[rng.random((T, k)) < 0.2] = -1
    elif kind == "elsewhere":
        ids = np.full((T, k), start + L)
    elif kind == "twice":     # an expert listed more than once
        ids[:, -1] = ids[:, 0]
        ids[::2, k // 2] = ids[::2, 0]
    elif kind == "one":       # every token the same expert
        ids = np.tile(np.arange(start, start + k), (T, 1))
    elif kind == "garbage":
        ids[:, 0] = rng.choice([2 ** 31 - 1, -2 ** 31, -5, start - 1, start + L], T)
    return ids.astype(np.int32), (rng.random((T, k)) + 0.1).astype(np.float32)


def check(x, ids, w, start, weights, w1, w2, h, out, add):
    """h [T, k, I] and out [T, H] of a call against float64."""
    T, k = ids.shape
    L, H, I = weights.num_local, weights.hidden, weights.inter
    x64, h64 = x.double(), h.double()
    ref = torch.zeros((T, H), dtype=torch.float64, device=DEV) if add is None else add.double()
    size, experts = ref.abs(), 0
    for e in sorted({int(i) - start for i in ids.flatten() if 0 <= int(i) - start < L}):
        at = [(t, int(np.nonzero(ids[t] - start == e)[0][0]), float(w[t][ids[t] - start == e].astype(np.float64).sum()))
              for t in range(T) if (ids[t] - start == e).any()]
        t, j = torch.tensor([a[0] for a in at], device=DEV), torch.tensor([a[1] for a in at], device=DEV)
        gs = weights.w1_gs[e].double().reshape(-1)
        W = values(w1[0][e], w1[1][e])
        gu = (x64[t] @ W.T.contiguous()) * torch.cat([gs[:1].expand(I), gs[-1:].expand(I)])
        terms = (x64[t].abs() @ W.abs().T.contiguous()) * torch.cat([gs[:1].expand(I), gs[-1:].expand(I)])
        err = STEP * (H / 16 + 26) * terms
        g, u = gu[:, :I], gu[:, I:]
        want = torch.nn.functional.silu(g) * u
        # through |silu'| <= 1.1 and |silu| <= |g|; silu's own roundings, of which e^-g has |g| times as many
        tol = 1.1 * err[:, :I] * (u.abs() + err[:, I:]) + g.abs() * err[:, I:] + (16 + 4 * g.abs()) * EPS32 * want.abs()
        got = h64[t, j]
        worst = ((got - want).abs() - tol * (1 + HALF_BF16) - HALF_BF16 * want.abs() - 2.0 ** -120).max()
        assert worst <= 0, ("h", e, float(worst))
        W = values(w2[0][e], w2[1][e]) * weights.w2_gs[e].double()
        wt = torch.tensor([a[2] for a in at], dtype=torch.float64, device=DEV)[:, None]
        ref.index_add_(0, t, (got @ W.T.contiguous()) * wt)
        size.index_add_(0, t, (got.abs() @ W.abs().T.contiguous()) * wt.abs())
        experts += 1
    tol = STEP * (I / 16 + 32 + min(k, experts) + k) * size
    worst = ((out.double() - ref).abs() - tol * (1 + HALF_BF16) - HALF_BF16 * ref.abs()).max()
    assert worst <= 0, ("out", float(worst))


CASES = [
    # T, k, E, L, start, H, I, dual, add, choices
    (1, 1, 1, 1, 0, 128, 128, False, False, "plain"),
    (1, 8, 32, 32, 0, 1024, 512, False, True, "plain"),
    (1, 8, 64, 8, 24, 512, 384, True, False, "plain"),
    (2, 4, 16, 16, 0, 384, 128, True, True, "twice"),
    (5, 4, 64, 16, 16, 512, 384, False, False, "masked"),
    (31, 2, 3, 3, 0, 256, 640, False, True, "plain"),
    (32, 8, 8, 8, 0, 256, 128, True, False, "plain"),
    (33, 3, 9, 4, 2, 640, 256, False, True, "garbage"),
    (64, 8, 384, 48, 96, 1024, 384, False, False, "masked"),
    (64, 4, 4, 4, 0, 256, 256, False, True, "one"),
    (64, 1, 2, 1, 1, 128, 2048, True, False, "plain"),
    (64, 64, 100, 70, 20, 128, 128, False, True, "twice"),
    (64, 8, 4096, 4096, 0, 128, 128, False, False, "plain"),
    (7, 5, 12, 6, 3, 7168, 128, False, True, "elsewhere"),
    (40, 6, 200, 100, 50, 128, 1152, True, True, "twice"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_layer(nv, case):
    T, k, E, L, start, H, I, dual, with_add, kind = case
    weights, w1, w2, g = layer(nv, L, H, I, dual, T + L)
    ids, w = choices(kind, T, k, E, start, L, T)
    x = torch.randn(T, H, device=DEV, generator=g).bfloat16()
    add = torch.randn(T, H, device=DEV, generator=g).bfloat16() if with_add else None
    ws, ws_ok = guarded((nv.nvfp4_moe_few_ws_bytes(T, k, H, I, L),), torch.uint8, 0x7F)
    ws.fill_(0xFF)                                    # NaN wherever a row that no choice wrote is read
    out, intact = guarded((T, H), torch.bfloat16, 7.0)
    nv.nvfp4_moe_forward_few(weights, x, to_dev(ids), to_dev(w), start, add=add, out=out, ws=ws)
    assert intact() and ws_ok()
    h = ws[:T * k * I * 2].view(torch.bfloat16).view(T, k, I)
    check(x, ids, w, start, weights, w1, w2, h, out, add)
    # again on another workspace, and in place of what is added
    assert torch.equal(nv.nvfp4_moe_forward_few(weights, x, to_dev(ids), to_dev(w), start, add=add), out)
    if with_add:
        nv.nvfp4_moe_forward_few(weights, x, to_dev(ids), to_dev(w), start, add=add, out=add)
        assert torch.equal(add, out)


@pytest.mark.parametrize("n", [1, 3, 4, 5, 7, 8, 9, 16, 17, 31, 32, 33, 40, 63, 64])
def test_tokens_of_an_expert(nv, n):
    """n of 64 tokens on one expert, the rest on another or none, in the places where they fall."""
    T, k, L, H, I = 64, 2, 5, 640, 384
    weights, w1, w2, g = layer(nv, L, H, I, True, 100 + n)
    rng = np.random.default_rng(n)
    ids = np.full((T, k), -1, np.int32)
    on = rng.permutation(T)[:n]
    ids[on, rng.integers(0, k, n)] = 3
    ids[rng.random((T, k)) < 0.2] = 9          # of another rank
    off = np.setdiff1d(np.arange(T), on)
    ids[off[::3], 0] = 1
    ids[on, 0] = np.where(ids[on, 1] == 3, 0, 3)
    w = (rng.random((T, k)) + 0.1).astype(np.float32)
    x = torch.randn(T, H, device=DEV, generator=g).bfloat16()
    ws = torch.full((nv.nvfp4_moe_few_ws_bytes(T, k, H, I, L),), 0xFF, dtype=torch.uint8, device=DEV)
    out = nv.nvfp4_moe_forward_few(weights, x, to_dev(ids), to_dev(w), 0, ws=ws)
    assert int((ids == 3).any(1).sum()) == n
    check(x, ids, w, 0, weights, w1, w2, ws[:T * k * I * 2].view(torch.bfloat16).view(T, k, I), out, None)


def test_oracle_of_the_layer(nv):
    """The NumPy oracle on one small layer, end to end (the rounding of h within half a step of BF16)."""
    T, k, L, H, I = 3, 2, 4, 128, 128
    weights, w1, w2, g = layer(nv, L, H, I, False, 3)
    ids, w = choices("plain", T, k, L, 0, L, 1)
    x = torch.randn(T, H, device=DEV, generator=g).bfloat16()
    full = [np.stack([O.dequantize(q[e].cpu().numpy(), sf[e].cpu().numpy()) * float(gs[e]) for e in range(L)])
            for (q, sf), gs in ((w1, weights.w1_gs), (w2, weights.w2_gs))]
    ref, size = F.forward(x.double().cpu().numpy(), ids, w, 0, *full)
    got = nv.nvfp4_moe_forward_few(weights, x, to_dev(ids), to_dev(w), 0).double().cpu().numpy()
    # h may round the other way next to a half: one BF16 step of it
    assert (np.abs(got - ref) <= 2.02 * HALF_BF16 * size + HALF_BF16 * np.abs(ref)).all()


def test_one_bad_token(nv):
    """Infinities and NaN stay with the token that holds them; experts that nobody chose are not read."""
    T, k, L, H, I = 20, 3, 8, 256, 256
    weights, w1, w2, g = layer(nv, L, H, I, False, 9)
    ids, w = choices("plain", T, k, L - 1, 0, L - 1, 2)      # nobody takes the last expert
    x = torch.randn(T, H, device=DEV, generator=g).bfloat16()
    clean = nv.nvfp4_moe_forward_few(weights, x, to_dev(ids), to_dev(w), 0)
    weights.w1[L - 1] = 0x7F
    weights.w2[L - 1] = 0x7F
    weights.w2_gs[L - 1] = float("nan")
    x[4, 7], x[11, 200] = float("nan"), float("inf")
    got = nv.nvfp4_moe_forward_few(weights, x, to_dev(ids), to_dev(w), 0)
    rest = [t for t in range(T) if t not in (4, 11)]
    assert torch.equal(got[rest], clean[rest])
    assert torch.isnan(got[4]).all() and not torch.isfinite(got[11]).all()


def test_close_to_the_layer(nv):
    """Against nvfp4_moe_forward on prepared weights: the same layer but for the activations' NVFP4."""
    T, k, L, H, I = 24, 4, 16, 512, 384
    g = torch.Generator(device=DEV).manual_seed(4)
    wg, wu, wd = (torch.randn(s, device=DEV, generator=g).mul(0.05).bfloat16() for s in ((L, I, H), (L, I, H), (L, H, I)))
    x = torch.randn(T, H, device=DEV, generator=g).bfloat16()
    ids, w = (to_dev(v) for v in choices("plain", T, k, 2 * L, 0, L, 5))
    for fold in (True, False):
        weights = nv.prepare_weights(wg, wu, wd, fold=fold)
        few, full = (f(weights, x, ids, w, 4).float() for f in (nv.nvfp4_moe_forward_few, nv.nvfp4_moe_forward))
        assert torch.nn.functional.cosine_similarity(few.flatten(), full.flatten(), 0) > 0.98
        exact = torch.zeros(T, H, device=DEV, dtype=torch.float64)
        for t in range(T):
            for j in range(k):
                e = int(ids[t, j]) - 4
                if 0 <= e < L:
                    v = x[t].double()
                    exact[t] += float(w[t, j]) * (wd[e].double() @ (torch.nn.functional.silu(wg[e].double() @ v) * (wu[e].double() @ v)))
        err = [float((v.double() - exact).norm()) for v in (few, full)]
        assert err[0] < err[1]     # only the weights are rounded


def test_empty_and_refused(nv):
    weights, *_ = layer(nv, 2, 128, 128, False, 1)
    x = torch.zeros(0, 128, dtype=torch.bfloat16, device=DEV)
    ids, w = torch.zeros(0, 2, dtype=torch.int32, device=DEV), torch.zeros(0, 2, device=DEV)
    assert nv.nvfp4_moe_forward_few(weights, x, ids, w, 0).shape == (0, 128)
    T = nv.nvfp4_moe_few_max_tokens() + 1
    x = torch.zeros(T, 128, dtype=torch.bfloat16, device=DEV)
    ids, w = torch.zeros(T, 2, dtype=torch.int32, device=DEV), torch.zeros(T, 2, device=DEV)
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_moe_forward_few(weights, x, ids, w, 0)
    for bad in (dict(x=x[:5].float()), dict(x=x[:5, :64].contiguous()), dict(ids=ids[:4]), dict(w=w[:5, :1].contiguous()),
                dict(add=x[:4]), dict(out=x[:4]), dict(ids=ids[:5].long())):
        call = dict(x=x[:5], ids=ids[:5], w=w[:5], add=None, out=None)
        call.update(bad)
        with pytest.raises(ValueError):
            nv.nvfp4_moe_forward_few(weights, call["x"], call["ids"], call["w"], 0, add=call["add"], out=call["out"])
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_moe_forward_few(weights, x[:5], ids[:5], w[:5], 0, ws=torch.zeros(64, dtype=torch.uint8, device=DEV))


def test_in_place(nv):
    """The output over the input, and over what is added, with the down products whole and in parts."""
    for T, k, L, H, I in ((3, 2, 8, 256, 128), (64, 8, 40, 512, 512)):
        weights, *_, g = layer(nv, L, H, I, False, 8)
        x, add = (torch.randn(T, H, device=DEV, generator=g).bfloat16() for _ in range(2))
        ids, w = (to_dev(v) for v in choices("plain", T, k, L, 0, L, 8))
        want = nv.nvfp4_moe_forward_few(weights, x, ids, w, 0, add=add)
        for over in (x, add):
            given = dict(x=x.clone(), add=add.clone())
            out = given["x" if over is x else "add"]
            nv.nvfp4_moe_forward_few(weights, given["x"], ids, w, 0, add=given["add"], out=out)
            assert torch.equal(out, want)
    assert nv.nvfp4_moe_few_ws_bytes(64, 8, 512, 512, 40) > 64 * 8 * 512 * 2 >= nv.nvfp4_moe_few_ws_bytes(3, 2, 256, 128, 8)


def test_in_a_graph(nv):
    """Captured, then replayed with other choices in the same buffers."""
    T, k, L, H, I = 9, 4, 12, 256, 256
    weights, *_, g = layer(nv, L, H, I, True, 6)
    x, out = torch.randn(T, H, device=DEV, generator=g).bfloat16(), torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    sets = [[to_dev(v) for v in choices(kind, T, k, 16, 2, L, i)] for i, kind in enumerate(("plain", "masked", "one", "elsewhere"))]
    ids, w = sets[0][0].clone(), sets[0][1].clone()
    ws = torch.empty(nv.nvfp4_moe_few_ws_bytes(T, k, H, I, L), dtype=torch.uint8, device=DEV)
    nv.nvfp4_moe_forward_few(weights, x, ids, w, 2, out=out, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.nvfp4_moe_forward_few(weights, x, ids, w, 2, out=out, ws=ws)
    for i, wt in sets + sets[:2]:
        ids.copy_(i)
        w.copy_(wt)
        ws.fill_(0xFF)
        out.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, nv.nvfp4_moe_forward_few(weights, x, i, wt, 2))
