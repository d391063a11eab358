"""Sizes from which inputs are read, and outputs written, past the caches: bit for bit what their parts give, which the
other tests hold to the oracle."""
import pytest
import torch

from _block_cases import DEV, EPS32

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def nv():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import nvfp4_quantized_moe_amd as nv
    return nv


@pytest.mark.parametrize("M,K,dtype", [(2344, 7176, BF16), (16781, 1000, BF16), (1171, 7176, F32), (40001, 216, F32)])
def test_codes(nv, M, K, dtype):
    assert M * K * (2 if dtype is BF16 else 4) >= 32 << 20
    x = (torch.randn(M, K, device=DEV) * torch.randn(K, device=DEV).exp()).to(dtype)
    for rule in (nv.MX_SCALE_FLOOR, nv.MX_SCALE_CEIL):
        q, s, qt, st = nv.mxfp4_quantize(x, nv.MX_BOTH, rule=rule)
        for got, want in zip(nv.mxfp4_quantize(x, nv.MX_ROWS, rule=rule) + nv.mxfp4_quantize(x, nv.MX_COLUMNS, rule=rule),
                             (q, s, qt, st)):
            assert torch.equal(got, want)
        third = M // 3
        rows = [nv.mxfp4_quantize(p.contiguous(), rule=rule) for p in x.split(third)]
        assert torch.equal(q, torch.cat([p[0] for p in rows])) and torch.equal(s, torch.cat([p[1] for p in rows], 1))
        cut = K // 24 * 8
        cols = [nv.mxfp4_quantize(p.contiguous(), nv.MX_COLUMNS, rule=rule) for p in x.split(cut, 1)]
        assert torch.equal(qt, torch.cat([p[0] for p in cols])) and torch.equal(st, torch.cat([p[1] for p in cols], 1))


@pytest.mark.parametrize("with_add", [False, True])
@pytest.mark.parametrize("M,N,dtype,silu", [(16400, 4096, BF16, False), (16393, 8208, BF16, True), (8200, 4104, F32, False)])
def test_products(nv, M, N, dtype, silu, with_add):
    """Sums of 128 terms of few bits: exact in any order."""
    n = N // 2 if silu else N
    assert M * n * (2 if dtype is BF16 else 4) >= 128 << 20
    a, b = (torch.randint(0, 256, (r, 64), dtype=torch.uint8, device=DEV) for r in (M, N))
    sa, sb = (torch.full((1, r, 4), 125, dtype=torch.uint8, device=DEV) for r in (M, N))
    add = torch.randn(M, n, device=DEV).to(dtype) if with_add else None
    epilogue = nv.EPI_SILU_MUL if silu else nv.EPI_BF16
    d = nv.mxfp4_gemm(a, sa, b, sb, epilogue, add=add, dtype=dtype)
    for rows in torch.arange(M, device=DEV).split(64)[::37]:
        part = nv.mxfp4_gemm(a[rows], sa[:, rows].contiguous(), b, sb, epilogue, add=add[rows] if with_add else None, dtype=dtype)
        assert torch.equal(d[rows], part)
    if with_add:
        assert torch.equal(nv.mxfp4_gemm(a, sa, b, sb, epilogue, add=add, dtype=dtype, d=add), d)


@pytest.mark.parametrize("x_type", [BF16, F32])
@pytest.mark.parametrize("T,H", [(2340, 7176), (1030, 16384), (5000, 4096), (9000, 2048)])
def test_layer_norm(nv, T, H, x_type):
    assert T * H * 2 >= 32 << 20
    x, d_y = (torch.randn(T, H, device=DEV).to(x_type) for _ in range(2))
    res, d_r = (torch.randn(T, H, device=DEV).bfloat16() for _ in range(2))
    w, b = torch.randn(H, device=DEV), torch.randn(H, device=DEV)
    r, y, q, s = nv.moe_layer_norm(x, res, w, b, 0.75, mx_rule=nv.MX_SCALE_FLOOR)
    g = nv.moe_layer_norm_backward(d_y, d_r, r, w, b, 0.75)
    parts = [slice(i, min(i + T // 3, T)) for i in range(0, T, T // 3)]
    sums = [torch.zeros(H, dtype=torch.float64, device=DEV) for _ in range(2)]
    for p in parts:
        for got, want in zip(nv.moe_layer_norm(x[p], res[p], w, b, 0.75, mx_rule=nv.MX_SCALE_FLOOR), (r[p], y[p], q[p], s[:, p])):
            assert torch.equal(got, want)
        h = nv.moe_layer_norm_backward(d_y[p], d_r[p], r[p], w, b, 0.75)
        assert torch.equal(h["d_x"], g["d_x"][p]) and torch.equal(h["d_residual"], g["d_residual"][p])
        for total, n in zip(sums, ("d_w", "d_b")):
            total += h[n].double()
    # both sides: n within 192 steps of itself, and at most T / 256 + 64 additions behind a term
    v = r.double()
    n = (v - v.mean(1, keepdim=True)) / (v.var(1, correction=0, keepdim=True) + 1e-5).sqrt()
    for name, total, terms in (("d_w", sums[0], (n.abs() + 1) * d_y.double().abs()), ("d_b", sums[1], d_y.double().abs())):
        tol = 2 * (256 + T / 256) * EPS32 * terms.sum(0)
        assert ((g[name].double() - total).abs() <= tol).all()
    out, old = x.clone(), res.clone()
    r2, y2 = nv.moe_layer_norm(out, old, w, b, 0.75, residual_out=old, y=out)
    assert torch.equal(r2, r) and torch.equal(y2, y)
    h = nv.moe_layer_norm_backward(d_y, d_r, r, w, b, 0.75, d_x=d_y, d_residual=d_r)
    assert h["d_x"] is d_y and all(torch.equal(h[k], g[k]) for k in g)


def test_longest_rows(nv):
    """262144 elements along a row of codes, either way, and products over all of them: sums of random signs stay far
    from the 2^22 up to which quarters are exact."""
    n = 262144
    x = torch.randn(3, n, device=DEV).bfloat16()
    q, s = nv.mxfp4_quantize(x)
    half = [nv.mxfp4_quantize(p.contiguous()) for p in x.chunk(2, 1)]
    assert torch.equal(q, torch.cat([p[0] for p in half], 1)) and torch.equal(s, torch.cat([p[1] for p in half]))
    x = torch.randn(n, 8, device=DEV).bfloat16()
    q, s, qt, st = nv.mxfp4_quantize(x, nv.MX_BOTH)
    half = [nv.mxfp4_quantize(p, nv.MX_BOTH) for p in x.chunk(2)]
    assert torch.equal(qt, torch.cat([p[2] for p in half], 1)) and torch.equal(st, torch.cat([p[3] for p in half]))
    assert torch.equal(q, torch.cat([p[0] for p in half])) and torch.equal(s, torch.cat([p[1] for p in half], 1))
    g = torch.Generator(device=DEV).manual_seed(1)
    for M, N in ((1, 8), (3, 4096), (40, 16), (300, 136)):
        a, b = (torch.randint(0, 256, (r, n // 2), dtype=torch.uint8, device=DEV, generator=g) for r in (M, N))
        sa, sb = (torch.full((n // 128, r, 4), 127, dtype=torch.uint8, device=DEV) for r in (M, N))
        A, B = nv.mxfp4_dequantize(a, sa).double(), nv.mxfp4_dequantize(b, sb).double()
        ref = A @ B.T.contiguous()
        assert ref.abs().max() < 2.0 ** 18
        assert torch.equal(nv.mxfp4_gemm(a, sa, b, sb, dtype=F32).double(), ref), (M, N)
        got = nv.mxfp4_gemm(a, sa, b, sb, add=torch.ones(M, N, device=DEV).bfloat16())
        assert torch.equal(got, (ref + 1).float().bfloat16())
