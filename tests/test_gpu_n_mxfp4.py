"""MXFP4 quantisation, its inverse and the products against the oracle.

Codes, scales and values are exact. A product's terms are exact in float32 (two
significant bits each); its sum rounds at most once per addition, and one of
its K additions follows at most K / 64 + 128 + parts others (64 or 128 terms of
an instruction in any order, the instructions of a wave one after the other, the
waves and parts of K), each within one float32 step of the terms' sum.
"""
import numpy as np
import pytest
import torch

import oracle.int8 as I8
import oracle.mxfp4 as MX
from _block_cases import DEV, EPS32, HALF_BF16, as_stored, guarded, to_dev, torch_dtype

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import nvfp4_quantized_moe_amd as nv
    return nv


def values(M, K, kind, dtype, seed=0):
    rng = np.random.default_rng(1000 * M + K + seed)
    x = rng.standard_normal((M, K)) * np.exp(rng.standard_normal(K) * 0.5)
    if kind == "ties":        # halves of the grid at many scales, signed zeros
        x = rng.choice([0, 0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7], (M, K))
        x *= rng.choice([-1.0, 1.0], (M, K)) * np.exp2(np.repeat(rng.integers(-30, 30, (M, -(-K // 32))), 32, 1)[:, :K])
    elif kind == "sizes":     # blocks from subnormals to the largest numbers, some of zeros
        x = rng.standard_normal((M, K)) * np.exp2(np.repeat(rng.integers(-150, 126, (M, -(-K // 32))), 32, 1)[:, :K])
        x = np.clip(x, -3.3e38, 3.3e38)
        x[:, 32:64] = 0.0
    return as_stored(x, dtype)


SIZES = [(1, 8), (1, 7168), (3, 40), (5, 1000), (64, 7168), (33, 1040), (128, 128), (129, 136), (257, 520), (700, 264),
         (4099, 72), (2047, 2888), (33001, 72)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["plain", "ties", "sizes"])
@pytest.mark.parametrize("M,K", SIZES)
def test_codes(nv, M, K, kind, dtype):
    rule = (M + K // 8) % 2
    x = values(M, K, kind, dtype)
    dev = to_dev(x.astype(np.float32), torch_dtype(dtype))
    Mp, Kp = nv.mxfp4_padded(M), nv.mxfp4_padded(K)
    rows, cols = MX.quantize(x, rule), MX.quantize(x.T, rule)
    for way in (nv.MX_ROWS, nv.MX_COLUMNS, nv.MX_BOTH):
        q, q_ok = guarded((M, Kp // 2), torch.uint8, 0x5A)
        s, s_ok = guarded((Kp // 128, M, 4), torch.uint8, 0x5A)
        qt, qt_ok = guarded((K, Mp // 2), torch.uint8, 0x5A)
        st, st_ok = guarded((Mp // 128, K, 4), torch.uint8, 0x5A)
        given = {}
        if way & nv.MX_ROWS:
            given.update(q=q, scale=s)
        if way & nv.MX_COLUMNS:
            given.update(q_t=qt, scale_t=st)
        got = nv.mxfp4_quantize(dev, way, rule=rule, **given)
        assert q_ok() and s_ok() and qt_ok() and st_ok()
        want = (rows if way & nv.MX_ROWS else ()) + (cols if way & nv.MX_COLUMNS else ())
        assert len(got) == len(want)
        for g, w in zip(got, want):
            assert np.array_equal(g.cpu().numpy(), w), (way, g.shape)
    # and back, whole and cut to the columns there were
    v = MX.dequantize(*rows)
    full = nv.mxfp4_dequantize(q, s, torch.float32)
    assert np.array_equal(full.double().cpu().numpy(), v)
    for t in (torch.bfloat16, torch.float32):
        out, intact = guarded((M, K), t, 7.0)
        nv.mxfp4_dequantize(q, s, t, cols=K, out=out)
        assert intact() and np.array_equal(out.double().cpu().numpy(), v[:, :K])
    back = nv.mxfp4_dequantize(qt, st, torch_dtype(dtype), cols=M)   # rows of an odd length
    assert np.array_equal(back.double().cpu().numpy(), MX.dequantize(*cols)[:, :M])


def test_every_bf16(nv):
    """All finite BF16 patterns, each in a block whose largest is within a factor of 2^9."""
    bits = np.arange(65536, dtype=np.uint16)
    x = (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    x = x[np.isfinite(x)]
    x = x[np.argsort(np.abs(x), kind="stable")].reshape(-1, 32)
    for rule in (MX.FLOOR, MX.CEIL):
        q, s = nv.mxfp4_quantize(to_dev(x.astype(np.float32), torch.bfloat16), rule=rule)
        ref = MX.quantize(x, rule)
        assert np.array_equal(q.cpu().numpy(), ref[0]) and np.array_equal(s.cpu().numpy(), ref[1])


def test_every_value(nv):
    """All codes at all scales, the NaN scale and values past the range among them."""
    q = np.tile(np.arange(256, dtype=np.uint8), (256, 1))[:, :64].copy()
    q[:, 16:32] = np.arange(16) * 17
    s = np.tile(np.arange(256, dtype=np.uint8)[None, :, None], (1, 1, 4))
    ref = MX.dequantize(q, s)
    with np.errstate(over="ignore"):
        ref = ref.astype(np.float32)
    for t in (torch.bfloat16, torch.float32):
        got = nv.mxfp4_dequantize(to_dev(q), to_dev(s), t).float().cpu().numpy()
        assert np.array_equal(got, ref, equal_nan=True)


def test_not_finite(nv):
    """A block with an infinity or NaN is NaN in both directions, its neighbours are what they were, and a product has
    NaN in that row alone."""
    x = values(70, 256, "plain", "f32")
    ref = x.copy()
    for (r, c), bad in {(3, 40): np.inf, (20, 100): -np.inf, (66, 255): np.nan}.items():
        x[r, c] = bad
        ref[r, c] = bad
    for t in (torch.bfloat16, torch.float32):
        dev = to_dev(x.astype(np.float32), t)
        xs = dev.double().cpu().numpy()
        q, s, qt, st = nv.mxfp4_quantize(dev, nv.MX_BOTH)
        for (a, b), w in (((q, s), MX.quantize(xs)), ((qt, st), MX.quantize(xs.T))):
            assert np.array_equal(b.cpu().numpy(), w[1])
            whole = np.repeat(w[1].transpose(1, 0, 2).reshape(len(w[0]), -1) != 255, 16, 1)
            assert np.array_equal(a.cpu().numpy()[whole], w[0][whole])
        b = MX.quantize(values(64, 256, "plain", "bf16", 1))
        for rows in (slice(0, 70), slice(3, 4), slice(2, 22)):
            xq, xsc = q[rows].contiguous(), s[:, rows].contiguous()
            d = nv.mxfp4_gemm(xq, xsc, to_dev(b[0]), to_dev(b[1]))
            nan_rows = torch.isnan(d).all(1).cpu().numpy()
            assert np.array_equal(nan_rows, np.isin(np.arange(70)[rows], [3, 20, 66]))
            assert not torch.isnan(d[torch.from_numpy(~nan_rows).to(DEV)]).any()


SHAPES = [(1, 8, 128), (1, 4096, 7168), (2, 16, 256), (5, 1000, 1152), (16, 4096, 7168), (17, 264, 7168), (33, 40, 384),
          (64, 4096, 7168), (63, 7168, 2048), (33, 72, 8320), (64, 520, 16384), (100, 1096, 7168), (65, 128, 128),
          (16, 64, 65536), (64, 4096, 16384), (128, 256, 65536), (333, 1000, 1152), (500, 520, 384), (1030, 2056, 1280),
          (2048, 2048, 256), (2049, 4104, 512), (4100, 1536, 128)]


def operands(M, N, K, seed):
    rng = np.random.default_rng(seed)
    a, b = rng.integers(0, 256, (M, K // 2), dtype=np.uint8), rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    a_s, b_s = rng.integers(122, 132, (K // 128, M, 4), dtype=np.uint8), rng.integers(116, 124, (K // 128, N, 4), dtype=np.uint8)
    return a, a_s, b, b_s, rng


def product(a, a_s, b, b_s):
    """(float64 product, the sum of its terms' magnitudes), on the GPU in float64."""
    A, B = (to_dev(MX.dequantize(q, s)) for q, s in ((a, a_s), (b, b_s)))
    return (A @ B.T.contiguous()).cpu().numpy(), (A.abs() @ B.abs().T.contiguous()).cpu().numpy()


def chain(K):
    return K / 64 + 128 + 64


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("with_add", [False, True])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(nv, M, N, K, with_add, dtype):
    a, a_s, b, b_s, rng = operands(M, N, K, 1)
    t = torch_dtype(dtype)
    add = as_stored(rng.standard_normal((M, N)) * 3, dtype) if with_add else np.zeros((M, N))
    d, intact = guarded((M, N), t, 7.0)
    call = [to_dev(v) for v in (a, a_s, b, b_s)]
    extra = to_dev(add.astype(np.float32), t) if with_add else None
    nv.mxfp4_gemm(*call, d=d, dtype=t, add=extra)
    assert intact()
    ref, terms = product(a, a_s, b, b_s)
    ref = ref + add
    got = d.double().cpu().numpy()
    tol = 2 * EPS32 * (chain(K) * terms + np.abs(add)) * (1 + HALF_BF16) + (HALF_BF16 if dtype == "bf16" else EPS32) * np.abs(ref)
    assert (np.abs(got - ref) <= tol).all(), float(np.max(np.abs(got - ref) / np.maximum(tol, 1e-30)))
    again = nv.mxfp4_gemm(*call, dtype=t, add=extra)
    assert torch.equal(again, d)
    if with_add:
        nv.mxfp4_gemm(*call, dtype=t, add=extra, d=extra)
        assert torch.equal(extra, d)


@pytest.mark.parametrize("with_add", [False, True])
@pytest.mark.parametrize("M,N,K", [s for s in SHAPES if s[1] % 16 == 0])
def test_product_silu(nv, M, N, K, with_add):
    a, a_s, b, b_s, rng = operands(M, N, K, 2)
    b_s -= int(np.log2(K) / 2)   # gates of a few units
    inter = N // 2
    add = as_stored(rng.standard_normal((M, inter)) * 3, "bf16") if with_add else np.zeros((M, inter))
    d, intact = guarded((M, inter), torch.bfloat16, 7.0)
    nv.mxfp4_gemm(*(to_dev(v) for v in (a, a_s, b, b_s)), nv.EPI_SILU_MUL, d=d,
                  add=to_dev(add.astype(np.float32), torch.bfloat16) if with_add else None)
    assert intact()
    gu, terms = product(a, a_s, b, b_s)
    g, u = gu[:, :inter], gu[:, inter:]
    e = 2 * EPS32 * chain(K) * terms
    h = I8.silu_mul(g, u)
    ref = h + add
    # the sums' errors through |silu'| <= 1.1 and |silu| <= |g|, then the roundings of silu and the product
    tol = 1.1 * e[:, :inter] * (np.abs(u) + e[:, inter:]) + np.abs(g) * e[:, inter:]
    tol += (16 + 4 * np.abs(g)) * EPS32 * np.abs(h) + EPS32 * np.abs(ref)
    tol = tol * (1 + HALF_BF16) + HALF_BF16 * np.abs(ref) + 2.0 ** -120
    got = d.double().cpu().numpy()
    assert (np.abs(got - ref) <= tol).all(), float(np.max(np.abs(got - ref) / np.maximum(tol, 1e-30)))


def test_scales_at_their_ends(nv):
    """Scale codes from 0 to 254: products that leave float32's range at either end (under its normal numbers a term
    may count as 0)."""
    rng = np.random.default_rng(5)
    for M, N, K in ((4, 64, 128), (200, 72, 256), (1100, 264, 256)):
        a, b = rng.integers(0, 256, (M, K // 2), dtype=np.uint8), rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
        a_s, b_s = np.full((K // 128, M, 4), 127, np.uint8), np.full((K // 128, N, 4), 127, np.uint8)
        a_s[:, 0], a_s[:, 1], a_s[:, 2] = 0, 254, 30
        b_s[:, 0], b_s[:, 1], b_s[:, 2], b_s[:, 3] = 254, 0, 120, 230
        ref, terms = product(a, a_s, b, b_s)
        got = nv.mxfp4_gemm(*(to_dev(v) for v in (a, a_s, b, b_s)), dtype=torch.float32).double().cpu().numpy()
        inside = (terms < 2.0 ** 127)
        tol = 2 * EPS32 * chain(K) * terms + K * 2.0 ** -126
        assert (np.abs(got - ref) <= tol)[inside].all()
        assert not np.isnan(got[inside]).any()


def test_refused(nv):
    x = torch.zeros(4, 256, device=DEV)
    q, s, qt, st = nv.mxfp4_quantize(x, nv.MX_BOTH)
    add = torch.zeros(4, 8, device=DEV).bfloat16()
    for call in (lambda: nv.mxfp4_quantize(x, 0), lambda: nv.mxfp4_quantize(x, 4), lambda: nv.mxfp4_quantize(x.half()),
                 lambda: nv.mxfp4_quantize(x.T), lambda: nv.mxfp4_quantize(x.cpu()), lambda: nv.mxfp4_quantize(x[0]),
                 lambda: nv.mxfp4_quantize(x, q_t=qt), lambda: nv.mxfp4_quantize(x, scale_t=st),
                 lambda: nv.mxfp4_quantize(x, nv.MX_COLUMNS, q=q), lambda: nv.mxfp4_quantize(x, nv.MX_COLUMNS, scale=s),
                 lambda: nv.mxfp4_quantize(x, q=q[:3].clone()), lambda: nv.mxfp4_quantize(x, scale=s[:1].clone()),
                 lambda: nv.mxfp4_quantize(torch.zeros(262145, 8, device=DEV), nv.MX_COLUMNS),
                 lambda: nv.mxfp4_dequantize(q, s, torch.float16), lambda: nv.mxfp4_dequantize(q, s, cols=257),
                 lambda: nv.mxfp4_dequantize(q, s, cols=-1), lambda: nv.mxfp4_dequantize(q, s.reshape(4, 8)),
                 lambda: nv.mxfp4_dequantize(q[:, :32].contiguous(), s), lambda: nv.mxfp4_dequantize(q, st),
                 lambda: nv.mxfp4_gemm(q, s, qt, st), lambda: nv.mxfp4_gemm(q, None, q, s),
                 lambda: nv.mxfp4_gemm(q, s, q, s, add=add), lambda: nv.mxfp4_gemm(q, s, q, s, dtype=torch.int32)):
        with pytest.raises(ValueError):
            call()
    b, bs = nv.mxfp4_quantize(torch.zeros(8, 256, device=DEV))
    for call in (lambda: nv.mxfp4_quantize(x, rule=2), lambda: nv.mxfp4_quantize(torch.zeros(4, 12, device=DEV)),
                 lambda: nv.mxfp4_gemm(q, s, q, s), lambda: nv.mxfp4_gemm(q, s, b, bs, nv.EPI_SILU_MUL),
                 lambda: nv.mxfp4_gemm(q, s, b, bs, 7)):
        with pytest.raises(nv.NVFP4Error):
            call()
    for g in range(1, 4):   # addresses off 16 bytes
        off = torch.zeros(q.numel() + 16, dtype=torch.uint8, device=DEV)[4 * g:][:q.numel()].view(q.shape)
        with pytest.raises(nv.NVFP4Error):
            nv.mxfp4_quantize(x, q=off)
        with pytest.raises(nv.NVFP4Error):
            nv.mxfp4_gemm(off, s, b, bs)


def test_empty(nv):
    q, s, qt, st = nv.mxfp4_quantize(torch.empty((0, 40), dtype=torch.bfloat16, device=DEV), nv.MX_BOTH)
    assert q.shape == (0, 64) and s.shape == (1, 0, 4) and qt.shape == (40, 0) and st.shape == (0, 40, 4)
    b, bs = nv.mxfp4_quantize(torch.ones((8, 40), device=DEV))
    assert nv.mxfp4_gemm(q, s, b, bs).shape == (0, 8)
    # the weight gradient of an empty batch: zeros, or what there was
    for n in (40, 8):
        b, bs = torch.empty((n, 0), dtype=torch.uint8, device=DEV), torch.empty((0, n, 4), dtype=torch.uint8, device=DEV)
        assert not nv.mxfp4_gemm(qt, st, b, bs, dtype=torch.float32).any()
        so_far = torch.randn(40, n, device=DEV)
        assert torch.equal(nv.mxfp4_gemm(qt, st, b, bs, dtype=torch.float32, add=so_far), so_far)
    assert nv.mxfp4_dequantize(qt, st).shape == (40, 0)


@pytest.mark.parametrize("T,N,K", [(5, 24, 40), (130, 136, 264)])
def test_training_products(nv, T, N, K):
    """The three products of a linear layer's step against those of the quantised operands."""
    rng = np.random.default_rng(T)
    x, w, dy = (as_stored(rng.standard_normal(s), "bf16") for s in ((T, K), (N, K), (T, N)))
    X, W, DY = (nv.mxfp4_quantize(to_dev(v.astype(np.float32), torch.bfloat16), nv.MX_BOTH, rule=nv.MX_SCALE_CEIL)
                for v in (x, w, dy))
    val = {n: [MX.dequantize(*MX.quantize(m, MX.CEIL)) for m in (v, v.T)] for n, v in (("x", x), ("w", w), ("dy", dy))}
    for got, a, b in ((nv.mxfp4_gemm(*X[:2], *W[:2], dtype=torch.float32), val["x"][0], val["w"][0]),
                      (nv.mxfp4_gemm(*DY[:2], *W[2:], dtype=torch.float32), val["dy"][0], val["w"][1]),
                      (nv.mxfp4_gemm(*DY[2:], *X[2:], dtype=torch.float32), val["dy"][1], val["x"][1])):
        ref, terms = a @ b.T, np.abs(a) @ np.abs(b).T
        assert got.shape == ref.shape
        assert (np.abs(got.double().cpu().numpy() - ref) <= 2 * EPS32 * chain(a.shape[1]) * terms).all()


@pytest.mark.parametrize("T,K", [(5, 8200), (40, 8200), (300, 8200), (9, 32776), (70, 16648)])
def test_equal_in_a_graph(nv, T, K):
    """Captured and replayed on a dirty workspace, with eager work between the replays."""
    x = torch.randn(T, K, device=DEV).bfloat16()
    b, bs = nv.mxfp4_quantize(torch.randn(264, K, device=DEV))
    q, s = nv.mxfp4_quantize(x)
    d = torch.empty((T, 264), dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(max(256, nv.mxfp4_gemm_ws_bytes(T, 264, nv.mxfp4_padded(K))), dtype=torch.uint8, device=DEV)

    def step():
        nv.mxfp4_quantize(x, q=q, scale=s)
        nv.mxfp4_gemm(q, s, b, bs, d=d, ws=ws)
    step()
    torch.cuda.synchronize()
    first = d.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in (d, q, s, ws):
            t.fill_(0x7F if t.dtype == torch.uint8 else -3)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(d, first)
        assert nv.mxfp4_gemm(q, s, b, bs).equal(first)
