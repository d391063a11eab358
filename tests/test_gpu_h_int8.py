"""8-bit integer rows, products and the dense expert against the oracle.

Row codes and scales are exact. A product's integer sum is exact too; after it
come its conversion, the product of the scales, their product with the sum and
the addition, each one rounding of float32 (2^-24), then one of BF16 (2^-8).
"""
import numpy as np
import pytest
import torch

import oracle.int8 as I8
from _block_cases import DEV, EPS32, HALF_BF16, as_stored, guarded, to_dev, torch_dtype

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import nvfp4_quantized_moe_amd as nv
    return nv


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K,kind", [(1, 16, "plain"), (7, 1040, "plain"), (333, 7168, "plain"), (64, 2048, "halves"),
                                      (40, 528, "sizes"), (3, 65536, "plain"), (6, 64, "zeros")])
def test_rows(nv, M, K, kind, dtype):
    rng = np.random.default_rng(M + K)
    x = rng.standard_normal((M, K))
    if kind == "halves":      # multiples of amax / 254: quotients on and next to the halves
        x = rng.integers(-254, 255, (M, K)) / 254.0
        x[:, 0] = 1.0
        x *= np.exp2(rng.integers(-20, 20, (M, 1))) * rng.choice([1.0, 1.25, 1.7109375], (M, 1))
    elif kind == "sizes":     # from subnormals to near the largest
        x *= np.exp2(np.linspace(-146, 124, M))[:, None]
    elif kind == "zeros":
        x[::2] = 0.0
        x[1, :] = 0.0
        x[1, 5] = -3.0
    x = as_stored(x, dtype)
    q, q_ok = guarded((M, K), torch.int8, 99)
    s, s_ok = guarded((M,), torch.float32, 9.0)
    nv.int8_quantize_rows(to_dev(x.astype(np.float32), torch_dtype(dtype)), q, s)
    assert q_ok() and s_ok()
    ref_q, ref_s = I8.quantize_rows(x)
    assert np.array_equal(s.cpu().numpy(), ref_s)
    assert np.array_equal(q.cpu().numpy(), ref_q)


SHAPES = [(1, 8, 16), (1, 7168, 2048), (2, 16, 32), (5, 1000, 1040), (16, 4096, 7168), (17, 264, 7168), (33, 40, 144),
          (64, 4096, 7168), (63, 7168, 2048), (33, 72, 4112), (100, 1096, 7168), (65, 128, 128), (128, 256, 65536),
          (333, 1000, 1040), (500, 520, 272), (1030, 2056, 1168), (2048, 2048, 256), (2049, 4104, 400), (4100, 1536, 128)]


def operands(M, N, K, seed):
    rng = np.random.default_rng(seed)
    a, b = rng.integers(-127, 128, (M, K), dtype=np.int8), rng.integers(-127, 128, (N, K), dtype=np.int8)
    if K >= 65536:   # the largest sum there can be
        a[0], b[0], b[1] = 127, 127, -127
    a_s = (rng.random(M) * 0.02 + 1e-3).astype(np.float32)
    b_s = (rng.random(N) * 1e-3 + 1e-5).astype(np.float32)
    return a, a_s, b, b_s, rng


@pytest.mark.parametrize("with_add", [False, True])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(nv, M, N, K, with_add):
    a, a_s, b, b_s, rng = operands(M, N, K, 1)
    add = as_stored(rng.standard_normal((M, N)) * 3, "bf16") if with_add else np.zeros((M, N))
    d, intact = guarded((M, N), torch.bfloat16, 7.0)
    nv.int8_gemm(to_dev(a), to_dev(a_s), to_dev(b), to_dev(b_s), d=d,
                 add=to_dev(add.astype(np.float32), torch.bfloat16) if with_add else None)
    assert intact()
    ref = I8.gemm(a, a_s, b, b_s)
    terms, ref = np.abs(ref) + np.abs(add), ref + add
    got = d.double().cpu().numpy()
    tol = 4 * EPS32 * terms * (1 + HALF_BF16) + HALF_BF16 * np.abs(ref)
    assert (np.abs(got - ref) <= tol).all(), float(np.max(np.abs(got - ref) / np.maximum(tol, 1e-30)))


@pytest.mark.parametrize("with_add", [False, True])
@pytest.mark.parametrize("M,N,K", [s for s in SHAPES if s[1] % 16 == 0])
def test_product_silu(nv, M, N, K, with_add):
    a, a_s, b, b_s, rng = operands(M, N, K, 2)
    inter = N // 2
    b_s *= 300.0 / np.sqrt(K)
    add = as_stored(rng.standard_normal((M, inter)) * 3, "bf16") if with_add else np.zeros((M, inter))
    d, intact = guarded((M, inter), torch.bfloat16, 7.0)
    nv.int8_gemm(to_dev(a), to_dev(a_s), to_dev(b), to_dev(b_s), nv.EPI_SILU_MUL, d=d,
                 add=to_dev(add.astype(np.float32), torch.bfloat16) if with_add else None)
    assert intact()
    gu = I8.gemm(a, a_s, b, b_s)
    g, u = gu[:, :inter], gu[:, inter:]
    h = I8.silu_mul(g, u)
    ref = h + add
    got = d.double().cpu().numpy()
    # g and u carry 3 roundings each; g's reach e^-g as |g| times as many; exp 2, sum, quotient, product, addition
    tol = ((16 + 4 * np.abs(g)) * EPS32 * np.abs(h) + EPS32 * np.abs(ref)) * (1 + HALF_BF16) + HALF_BF16 * np.abs(ref)
    tol += 2.0 ** -120   # e^-g past float32's range
    assert (np.abs(got - ref) <= tol).all(), float(np.max(np.abs(got - ref) / np.maximum(tol, 1e-30)))


@pytest.mark.parametrize("T,H,I", [(1, 7168, 2048), (3, 64, 16), (40, 4112, 2064), (70, 5120, 80), (64, 1040, 528),
                                   (20, 4096, 4112), (200, 512, 256), (1100, 1024, 512)])
def test_dense_expert_is_its_steps(nv, T, H, I):
    """The forward equals its public steps bit for bit (each checked above), on a dirty workspace."""
    g = torch.Generator(device=DEV).manual_seed(T)
    wg, wu = (torch.randn(I, H, device=DEV, generator=g) * H ** -0.5 for _ in range(2))
    wd = torch.randn(H, I, device=DEV, generator=g) * I ** -0.5
    w = nv.prepare_int8_weights(wg, wu, wd)
    assert np.array_equal(w.w1_q[:I].cpu().numpy(), I8.quantize_rows(wg.double().cpu().numpy())[0])
    x = torch.randn(T, H, device=DEV, generator=g).bfloat16()
    add = torch.randn(T, H, device=DEV, generator=g).bfloat16()
    ws = torch.full((nv.int8_ffn_ws_bytes(T, H, I),), 0xA5, dtype=torch.uint8, device=DEV)
    for extra in (None, add):
        out, intact = guarded((T, H), torch.bfloat16, 7.0)
        nv.int8_ffn_forward(w, x, add=extra, out=out, ws=ws)
        assert intact()
        q, s = nv.int8_quantize_rows(x)
        h = nv.int8_gemm(q, s, w.w1_q, w.w1_scale, nv.EPI_SILU_MUL)
        hq, hs = nv.int8_quantize_rows(h)
        ref = nv.int8_gemm(hq, hs, w.w2_q, w.w2_scale, add=extra)
        assert torch.equal(out.view(torch.int16), ref.view(torch.int16))
    in_place = add.clone()
    nv.int8_ffn_forward(w, x, add=in_place, out=in_place)
    assert torch.equal(in_place, ref)
    # close to the unquantized expert: two int8 roundings of inputs and weights, each about 0.5 % of an element's rms
    full = (torch.nn.functional.silu(x.float() @ wg.T) * (x.float() @ wu.T)) @ wd.T + add.float()
    cos = torch.nn.functional.cosine_similarity(full.flatten(), ref.float().flatten(), 0)
    assert cos > 0.999


@pytest.mark.parametrize("H,I", [(4352, 2176), (1040, 528)])
def test_token_by_itself(nv, H, I):
    """A token's outputs have the same bits whatever else the call holds, though other kernels compute them."""
    T = 2300
    g = torch.Generator(device=DEV).manual_seed(H)
    w = nv.prepare_int8_weights(*(torch.randn(s, device=DEV, generator=g) * 0.03 for s in ((I, H), (I, H), (H, I))))
    x, add = (torch.randn(T, H, device=DEV, generator=g).bfloat16() for _ in range(2))
    q, s = nv.int8_quantize_rows(x)
    add_h = torch.randn(T, I, device=DEV, generator=g).bfloat16()
    whole = nv.int8_ffn_forward(w, x, add=add)
    whole_h = nv.int8_gemm(q, s, w.w1_q, w.w1_scale, nv.EPI_SILU_MUL, add=add_h)
    add_up = torch.randn(T, 2 * I, device=DEV, generator=g).bfloat16()
    whole_up = nv.int8_gemm(q, s, w.w1_q, w.w1_scale, add=add_up)
    for n in (1, 16, 17, 130, 500, 1200):
        assert torch.equal(nv.int8_ffn_forward(w, x[:n], add=add[:n]), whole[:n])
        assert torch.equal(nv.int8_gemm(q[:n], s[:n], w.w1_q, w.w1_scale, nv.EPI_SILU_MUL, add=add_h[:n]), whole_h[:n])
        assert torch.equal(nv.int8_gemm(q[:n], s[:n], w.w1_q, w.w1_scale, add=add_up[:n]), whole_up[:n])


def test_empty(nv):
    q, s = nv.int8_quantize_rows(torch.empty((0, 32), dtype=torch.bfloat16, device=DEV))
    b, bs = torch.ones((8, 32), dtype=torch.int8, device=DEV), torch.ones(8, device=DEV)
    assert nv.int8_gemm(q, s, b, bs).shape == (0, 8)


def test_equal_in_a_graph(nv):
    for T in (5, 300):
        w = nv.prepare_int8_weights(torch.randn(256, 512, device=DEV), torch.randn(256, 512, device=DEV),
                                    torch.randn(512, 256, device=DEV))
        x, add = torch.randn(T, 512, device=DEV).bfloat16(), torch.randn(T, 512, device=DEV).bfloat16()
        out = torch.empty_like(x)
        ws = torch.empty(nv.int8_ffn_ws_bytes(T, 512, 256), dtype=torch.uint8, device=DEV)
        nv.int8_ffn_forward(w, x, add, out, ws)
        torch.cuda.synchronize()
        first = out.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            nv.int8_ffn_forward(w, x, add, out, ws)
        for _ in range(3):
            out.fill_(-3)
            ws.fill_(0xA5)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, first)
