"""The layer norm, the MXFP4 products and the layer for a few tokens as a block uses them: one decode step, captured and
replayed; two of them at once on two streams; one training step of a projection; and past 2^31 elements."""
import ctypes

import numpy as np
import pytest
import torch

import oracle.layer_norm as LN
import oracle.mxfp4 as MX
from _block_cases import DEV, EPS32, as_stored, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import nvfp4_quantized_moe_amd as nv
    return nv


class Block:
    """Residual stream -> layer norm (with its codes) -> router, dense expert and routed experts -> residual stream."""

    def __init__(self, nv, T, H=512, I=256, E=16, k=3, seed=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.nv, self.k = nv, k
        rand = lambda *s, scale=0.05: (torch.randn(*s, device=DEV, generator=g) * scale).bfloat16()  # noqa: E731
        self.w = nv.prepare_weights(rand(E, I, H), rand(E, I, H), rand(E, H, I))
        self.router = nv.mxfp4_quantize(rand(E, H, scale=0.2))
        self.dense = nv.mxfp4_quantize(rand(2 * I, H)), nv.mxfp4_quantize(rand(H, I))
        self.ln = torch.randn(H, device=DEV, generator=g).abs(), torch.randn(H, device=DEV, generator=g)
        self.x, self.res = rand(T, H, scale=1.0), rand(T, H, scale=2.0)
        e = lambda shape, t: torch.empty(shape, dtype=t, device=DEV)  # noqa: E731
        b16, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
        Hp, Ip = nv.mxfp4_padded(H), nv.mxfp4_padded(I)
        self.b = dict(r=e((T, H), b16), y=e((T, H), b16), q=e((T, Hp // 2), u8), s=e((Hp // 128, T, 4), u8),
                      logits=e((T, E), f32), ids=e((T, k), torch.int32), wk=e((T, k), f32), up=e((T, I), b16),
                      uq=e((T, Ip // 2), u8), us=e((Ip // 128, T, 4), u8), dense=e((T, H), b16), out=e((T, H), b16),
                      r2=e((T, H), b16), y2=e((T, H), b16),
                      ws=e((max(256, nv.nvfp4_moe_few_ws_bytes(T, k, H, I, E)),), u8),
                      gws=e((max(256, nv.mxfp4_gemm_ws_bytes(T, 2 * I, Hp)),), u8))

    def step(self):
        nv, b = self.nv, self.b
        nv.moe_layer_norm(self.x, self.res, *self.ln, scale=0.5, mx_rule=nv.MX_SCALE_CEIL, residual_out=b["r"], y=b["y"],
                          y_q=b["q"], y_scale=b["s"])
        nv.mxfp4_gemm(b["q"], b["s"], *self.router, dtype=torch.float32, d=b["logits"], ws=b["gws"])
        nv.moe_gate_topk(b["logits"], self.k, topk_ids=b["ids"], topk_w=b["wk"])
        nv.mxfp4_gemm(b["q"], b["s"], *self.dense[0], nv.EPI_SILU_MUL, d=b["up"], ws=b["gws"])
        nv.mxfp4_quantize(b["up"], rule=nv.MX_SCALE_CEIL, q=b["uq"], scale=b["us"])
        nv.mxfp4_gemm(b["uq"], b["us"], *self.dense[1], d=b["dense"], ws=b["gws"])
        nv.nvfp4_moe_forward_few(self.w, b["y"], b["ids"], b["wk"], 0, add=b["dense"], out=b["out"], ws=b["ws"])
        nv.moe_layer_norm(b["out"], b["r"], *self.ln, scale=0.5, residual_out=b["r2"], y=b["y2"])

    RESULTS = ("r", "y", "q", "s", "logits", "ids", "wk", "up", "uq", "us", "dense", "out", "r2", "y2")

    def results(self):
        torch.cuda.synchronize()
        return {n: self.b[n].clone() for n in self.RESULTS}

    def spoil(self):
        for t in self.b.values():
            t.fill_(0x7F if t.dtype == torch.uint8 else -3)


def same(a, b):
    return [n for n in a if not torch.equal(a[n], b[n])]


@pytest.mark.parametrize("T", [1, 7, 33, 64])
def test_block(nv, T):
    """Each call's output from the call before it, in float64, and the whole in a graph."""
    B = Block(nv, T)
    B.step()
    got = B.results()
    f = {n: t.double().cpu().numpy() for n, t in got.items()}
    res, x = B.res.double().cpu().numpy(), B.x.double().cpu().numpy()
    w, b = (t.double().cpu().numpy() for t in B.ln)
    assert np.abs(f["r"] - (res + 0.5 * x)).max() <= 2.0 ** -8 * np.abs(f["r"]).max()
    y = LN.forward(f["r"], w, b)
    assert (np.abs(f["y"] - y) <= 2.0 ** -8 * np.abs(y) + 96 * EPS32 * (np.abs(y) + 4 * w + np.abs(b))).all()
    assert np.array_equal(got["q"].cpu().numpy(), MX.quantize(f["y"], MX.CEIL)[0])
    val = lambda q, s: MX.dequantize(q.cpu().numpy(), s.cpu().numpy())  # noqa: E731
    yq = val(got["q"], got["s"])
    chain = yq.shape[1] / 64 + 192
    logits = yq @ val(*B.router).T
    assert (np.abs(f["logits"] - logits) <= 2 * EPS32 * chain * (np.abs(yq) @ np.abs(val(*B.router)).T)).all()
    assert np.array_equal(np.sort(got["ids"].cpu().numpy(), 1), np.sort(torch.topk(got["logits"], B.k, dim=1).indices.cpu().numpy(), 1))
    alone = nv.nvfp4_moe_forward_few(B.w, got["y"], got["ids"], got["wk"], 0).double().cpu().numpy()
    assert (np.abs(f["out"] - alone - f["dense"]) <= 2.0 ** -7 * (np.abs(alone) + np.abs(f["dense"]))).all()
    B.step()
    assert not same(got, B.results())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.step()
    for _ in range(3):
        B.spoil()
        graph.replay()
        assert not same(got, B.results())


def test_two_streams_and_two_graphs(nv):
    """Two blocks with buffers of their own at once: eager on two streams, then as two graphs on two streams."""
    blocks = [Block(nv, 5, seed=1), Block(nv, 40, seed=2)]
    want = []
    for B in blocks:
        B.step()
        want.append(B.results())
    streams = [torch.cuda.Stream() for _ in blocks]
    graphs = []
    for B, s in zip(blocks, streams):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                B.step()
            graphs.append(g)
    torch.cuda.synchronize()
    for run in range(6):
        for B in blocks:
            B.spoil()
        torch.cuda.synchronize()
        for B, s, g in zip(blocks, streams, graphs):
            with torch.cuda.stream(s):
                if run % 2:
                    g.replay()
                else:
                    B.step()
        torch.cuda.synchronize()
        assert not any(same(w, B.results()) for w, B in zip(want, blocks))


def test_training_step(nv):
    """A projection behind a layer norm: forward and backward through the quantised operands, the weight's gradient
    added to what there was, against float64 on the same codes."""
    T, H, N = 130, 264, 136
    rng = np.random.default_rng(3)
    x, res, w, dy, dro = (as_stored(rng.standard_normal(s), "bf16") for s in ((T, H), (T, H), (N, H), (T, N), (T, H)))
    lw, lb = as_stored(1 + 0.2 * rng.standard_normal(H), "f32"), as_stored(rng.standard_normal(H), "f32")
    put = lambda a, t=torch.bfloat16: to_dev(a.astype(np.float32), t)  # noqa: E731
    lnw, lnb = put(lw, torch.float32), put(lb, torch.float32)
    r, y = nv.moe_layer_norm(put(x), put(res), lnw, lnb, scale=0.5)
    Y, W, DY = (nv.mxfp4_quantize(t, nv.MX_BOTH, rule=nv.MX_SCALE_CEIL) for t in (y, put(w), put(dy)))
    z = nv.mxfp4_gemm(*Y[:2], *W[:2])
    d_y = nv.mxfp4_gemm(*DY[:2], *W[2:])
    so_far = torch.randn(N, H, device=DEV)
    d_w = nv.mxfp4_gemm(*DY[2:], *Y[2:], dtype=torch.float32, add=so_far)
    g = nv.moe_layer_norm_backward(d_y, put(dro), r, lnw, lnb, scale=0.5)
    y64 = y.double().cpu().numpy()
    val = lambda a: MX.dequantize(*MX.quantize(a, MX.CEIL))  # noqa: E731
    for got, a, b, extra, step in ((z, val(y64), val(w), 0.0, 2.0 ** -8), (d_y, val(dy), val(w.T), 0.0, 2.0 ** -8),
                                   (d_w, val(dy.T), val(y64.T), so_far.double().cpu().numpy(), EPS32)):
        ref, terms = a @ b.T, np.abs(a) @ np.abs(b).T + np.abs(extra)
        tol = 2 * EPS32 * (a.shape[1] / 64 + 193) * terms * 1.01 + step * np.abs(ref + extra)
        assert (np.abs(got.double().cpu().numpy() - ref - extra) <= tol).all()
    ref = LN.backward(d_y.double().cpu().numpy(), dro, r.double().cpu().numpy(), lw, 0.5)
    for n, (value, terms) in ref.items():
        steps = 192 + (T / 256 + 64 if n in ("d_w", "d_b") else 0)
        tol = steps * EPS32 * terms * 1.01 + (2.0 ** -8 * np.abs(value) if n in ("d_x", "d_residual") else 0)
        assert (np.abs(g[n].double().cpu().numpy() - value) <= tol).all(), n


def test_norm_writes_codes_alone(nv):
    """The C entry without y: the codes are those of the y that is not stored."""
    for H, dt, code in ((264, torch.bfloat16, 0), (1000, torch.float32, 1)):
        x, w = torch.randn(9, H, device=DEV).to(dt), torch.randn(H, device=DEV)
        _, _, q, s = nv.moe_layer_norm(x, None, w, mx_rule=nv.MX_SCALE_CEIL)
        q2, s2 = torch.zeros_like(q), torch.zeros_like(s)
        st = nv._layer_norm(x.data_ptr(), code, None, code, 9, H, w.data_ptr(), None, 1.0, 1e-5, None, None,
                            nv.MX_SCALE_CEIL, q2.data_ptr(), s2.data_ptr(), ctypes.c_void_p(nv._stream()))
        torch.cuda.synchronize()
        assert st == 0 and torch.equal(q, q2) and torch.equal(s, s2)


def test_codes_past_32_bits(nv):
    """2.6e9 elements: the last rows and columns are those of the slice by itself."""
    M, K = 40064, 65536
    x = torch.empty(M, K, dtype=torch.bfloat16, device=DEV)
    for i in range(0, M, 4096):
        x[i:i + 4096] = torch.randn(min(4096, M - i), K, device=DEV)
    q, s, qt, st = nv.mxfp4_quantize(x, nv.MX_BOTH)
    tail = x[-256:].clone()
    a, b, c, d = nv.mxfp4_quantize(tail, nv.MX_BOTH)
    assert torch.equal(q[-256:], a) and torch.equal(s[:, -256:], b)
    assert torch.equal(qt[:, -128:], c) and torch.equal(st[-2:], d)
    only, sc = nv.mxfp4_quantize(x)
    assert torch.equal(only, q) and torch.equal(sc, s)
    del qt, st, only, sc
    assert torch.equal(nv.mxfp4_dequantize(q, s, out=x)[-256:], nv.mxfp4_dequantize(a, b))


def test_product_past_32_bits(nv):
    """Operands and an output of more than 2^31 bytes, with sums that float32 holds exactly in any order."""
    M, K, N = 70016, 65536, 64
    q = torch.zeros(M, K // 2, dtype=torch.uint8, device=DEV)
    q[:, ::64] = torch.randint(0, 256, (M, K // 128), dtype=torch.uint8, device=DEV)
    s = torch.full((K // 128, M, 4), 127, dtype=torch.uint8, device=DEV)
    b, bs = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=DEV), torch.full((K // 128, N, 4), 127, dtype=torch.uint8, device=DEV)
    d = nv.mxfp4_gemm(q, s, b, bs, dtype=torch.float32)
    for rows in (slice(0, 100), slice(M - 100, M)):
        part = nv.mxfp4_gemm(q[rows].contiguous(), s[:, rows].contiguous(), b, bs, dtype=torch.float32)
        A, Bm = nv.mxfp4_dequantize(q[rows].contiguous(), s[:, rows].contiguous(), torch.float32), nv.mxfp4_dequantize(b, bs, torch.float32)
        assert torch.equal(d[rows].double(), A.double() @ Bm.double().T.contiguous()) and torch.equal(part, d[rows])
    del q, s, d
    M, N, K = 36000, 32768, 128      # the output: 2.2e9 bytes in BF16
    a, b = (torch.randint(0, 256, (n, K // 2), dtype=torch.uint8, device=DEV) for n in (M, N))
    sa, sb = (torch.full((1, n, 4), 127, dtype=torch.uint8, device=DEV) for n in (M, N))
    d = nv.mxfp4_gemm(a, sa, b, sb)
    part = nv.mxfp4_gemm(a[-300:].contiguous(), sa[:, -300:].contiguous(), b, sb)
    assert torch.equal(d[-300:], part)


def test_layer_past_32_bits(nv):
    """Experts whose weights start beyond 2^31 bytes."""
    L, H, I, k = 200, 7168, 2048, 4
    w1 = torch.randint(0x28, 0x48, (L, 2 * I // 32, H // 128, 2304), dtype=torch.uint8, device=DEV)
    w2 = torch.randint(0x28, 0x48, (L, H // 32, I // 128, 2304), dtype=torch.uint8, device=DEV)
    gs = torch.full((L,), 1e-3, device=DEV)
    whole, last = nv.MoEWeights(w1, gs, w2, gs), nv.MoEWeights(w1[-k:].clone(), gs[-k:].clone(), w2[-k:].clone(), gs[-k:].clone())
    for T in (2, 20):
        x = torch.randn(T, H, device=DEV).bfloat16()
        ids = torch.arange(L - k, L, dtype=torch.int32, device=DEV).repeat(T, 1)
        w = torch.rand(T, k, device=DEV)
        assert torch.equal(nv.nvfp4_moe_forward_few(whole, x, ids, w, 0), nv.nvfp4_moe_forward_few(last, x, ids, w, L - k))


def test_norm_past_32_bits(nv):
    T, H = 300000, 8192
    x = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    for i in range(0, T, 32768):
        x[i:i + 32768] = torch.randn(min(32768, T - i), H, device=DEV)
    w, b = torch.randn(H, device=DEV), torch.randn(H, device=DEV)
    _, y = nv.moe_layer_norm(x, None, w, b)
    tail = x[-50:].clone()
    assert torch.equal(y[-50:], nv.moe_layer_norm(tail, None, w, b)[1])
    g = nv.moe_layer_norm_backward(y, None, x, w, b, residual=False)
    t = nv.moe_layer_norm_backward(y[-50:].clone(), None, tail, w, b, residual=False)
    assert torch.equal(g["d_x"][-50:], t["d_x"])


def test_outputs_of_its_own_in_a_graph(nv):
    """Outputs and workspaces that the calls allocate themselves, in a captured graph and in inference mode."""
    B = Block(nv, 6, seed=3)
    def chain():
        r, y, q, s = nv.moe_layer_norm(B.x, B.res, *B.ln, scale=0.5, mx_rule=nv.MX_SCALE_CEIL)
        logits = nv.mxfp4_gemm(q, s, *B.router, dtype=torch.float32)
        ids, wk = nv.moe_gate_topk(logits, B.k)
        up = nv.mxfp4_gemm(q, s, *B.dense[0], nv.EPI_SILU_MUL)
        dense = nv.mxfp4_gemm(*nv.mxfp4_quantize(up, rule=nv.MX_SCALE_CEIL), *B.dense[1])
        out = nv.nvfp4_moe_forward_few(B.w, y, ids, wk, 0, add=dense)
        g = nv.moe_layer_norm_backward(out, None, r, *B.ln, scale=0.5)
        return (r, y, q, s, logits, ids, wk, up, dense, out, *nv.moe_layer_norm(out, r, *B.ln, scale=0.5), *g.values())
    want = [t.clone() for t in chain()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain()
    for _ in range(3):
        for t in got:
            t.fill_(0x7F if t.dtype == torch.uint8 else -3)
        chain()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.inference_mode():
        out = chain()
        assert all(torch.equal(a, b) for a, b in zip(out, want)) and out[-1].is_inference()
    x = B.x.clone().requires_grad_()
    assert not nv.moe_layer_norm(x, None)[1].requires_grad and not nv.mxfp4_quantize(x)[0].requires_grad
