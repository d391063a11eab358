"""The operators around the expert FFN together, as one mixture-of-experts block uses them: pre-norm, gate, routed
experts in NVFP4, dense expert in 8-bit integers, post-norm and residual; and the training side of the gate and the
norms. Also what one call alone does not show: two streams at once, offsets past 32 bits, other devices' tensors."""
import numpy as np
import pytest
import torch

import oracle.gate as G
from _block_cases import DEV, EPS32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import nvfp4_quantized_moe_amd as nv
    return nv


class Block:
    """A small block: 16 of 32 experts local, hidden 512, inter 256, dense expert of inter 128."""

    def __init__(self, nv, seed=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.g, self.H, self.I, self.E, self.L, self.start, self.k = g, 512, 256, 32, 16, 8, 4
        r = lambda *s, scale=1.0: torch.randn(*s, device=DEV, generator=g) * scale  # noqa: E731
        self.r = r
        bf = lambda t: t.bfloat16()  # noqa: E731
        self.experts = nv.prepare_weights(bf(r(self.L, self.I, self.H, scale=0.05)), bf(r(self.L, self.I, self.H, scale=0.05)),
                                          bf(r(self.L, self.H, self.I, scale=0.05)), fold=False)
        self.dense = nv.prepare_int8_weights(r(128, self.H, scale=0.05), r(128, self.H, scale=0.05), r(self.H, 128, scale=0.05))
        self.w_gate = r(self.E, self.H, scale=0.05)
        self.bias = r(self.E, scale=0.05)
        self.w_pre, self.w_post, self.w_next = 1 + r(self.H, scale=0.1), 1 + r(self.H, scale=0.1), 1 + r(self.H, scale=0.1)
        self.gain = 0.5 + r(self.H, scale=0.1)

    def forward(self, nv, x, res, mask):
        res, y = nv.moe_block_norm(x, res, self.w_pre)
        logits = (y.float() @ self.w_gate.T).contiguous()
        ids, w = nv.moe_gate_topk(logits, self.k, nv.SCORE_SIGMOID, self.bias, mask, 8, 4, True, 2.0)
        routed = nv.nvfp4_moe_forward(self.experts, y, ids, w, self.start)
        out = nv.int8_ffn_forward(self.dense, y, add=routed)
        res2, y2 = nv.moe_block_norm(out, res, self.w_next, w_post=self.w_post, gate=self.gain, scale=0.8)
        return dict(res=res, y=y, logits=logits, ids=ids, w=w, routed=routed, out=out, res2=res2, y2=y2)


@pytest.mark.parametrize("T", [1, 33, 400])
def test_a_block_step(nv, T):
    b = Block(nv, T)
    x, res = b.r(T, b.H).bfloat16(), b.r(T, b.H, scale=2.0).bfloat16()
    mask = (torch.rand(T, device=DEV, generator=b.g) > 0.2).to(torch.uint8)
    mask[0] = 1
    d = b.forward(nv, x, res, mask)
    ids, w = G.gate_topk(d["logits"].cpu().double().numpy(), b.k, G.SIGMOID, b.bias.cpu().numpy(), mask.cpu().numpy(),
                         8, 4, True, 2.0)
    assert np.array_equal(d["ids"].cpu().numpy(), ids)
    # padding takes no part in the routed experts
    dead = mask == 0
    assert not d["routed"][dead].any()
    # the whole block in plain float64, with the experts' weights in float64: NVFP4 and int8 leave a few percent
    y = d["y"].double()
    dense = (torch.nn.functional.silu(y @ (b.dense.w1_q[:128].double() * b.dense.w1_scale[:128, None].double()).T)
             * (y @ (b.dense.w1_q[128:].double() * b.dense.w1_scale[128:, None].double()).T))
    dense = dense @ (b.dense.w2_q.double() * b.dense.w2_scale[:, None].double()).T
    diff = d["out"].double() - d["routed"].double()
    # int8 of y and of h: uniform errors of amax / 254 <= 1.7 % of an element's rms at 4.5 sigma, averaged over K
    assert torch.nn.functional.cosine_similarity(diff.flatten(), dense.flatten(), 0) > 0.998
    ref = b.gain.double() * 0.8 * d["out"].double() / torch.sqrt(d["out"].double().pow(2).mean(1, keepdim=True) + 1e-6) \
        * b.w_post.double() + d["res"].double()
    assert ((d["res2"].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 200 * EPS32 * 20).all()


def test_norm_output_feeds_the_expert_gemms(nv):
    """y as NVFP4 from the norm, then the separate steps, equals the static layer on y bit for bit."""
    b = Block(nv, 3)
    T = 400
    x, res = b.r(T, b.H).bfloat16(), b.r(T, b.H).bfloat16()
    _, y = nv.moe_block_norm(x, res, b.w_pre)
    logits = (y.float() @ b.w_gate.T).contiguous()
    ids, w = nv.moe_gate_topk(logits, b.k)
    gs = nv.calibrate_static_gs(b.experts, y, ids, w, b.start)
    want = nv.nvfp4_moe_forward_static(b.experts, y, ids, w, b.start, gs)
    _, y2, y_q, y_sf = nv.moe_block_norm(x, res, b.w_pre, gs=gs[:1])
    assert torch.equal(y, y2)
    tile = nv.nvfp4_moe_tile_m(T, b.k, b.L)
    r = nv.moe_route_slots(ids, w, b.start, b.L, tile)
    h_q, h_sf = nv.nvfp4_grouped_gemm_silu_nvfp4(y_q, y_sf, r["slot_token"], gs[:1].contiguous(), b.experts.w1,
                                                 b.experts.w1_gs, r["offsets"], r["tile_table"], T * b.k, tile,
                                                 gs[1:].clone())
    out = nv.nvfp4_grouped_gemm(h_q, h_sf, None, gs[1:].clone(), b.experts.w2, b.experts.w2_gs, r["offsets"],
                                r["tile_table"], T * b.k, tile)
    assert torch.equal(nv.moe_weighted_scatter(out, r["token_slot"], w), want)


def test_a_captured_block(nv):
    """The block captured once: every replay equals the eager step, also after new inputs and eager work between."""
    b = Block(nv, 5)
    T = 48
    x, res = b.r(T, b.H).bfloat16(), b.r(T, b.H).bfloat16()
    mask = torch.ones(T, dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.forward(nv, x, res, mask)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = b.forward(nv, x, res, mask)
    for i in range(4):
        x.copy_(b.r(T, b.H).bfloat16())
        mask[i] = 0
        want = b.forward(nv, x, res, mask)
        for t in got.values():
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n in ("ids", "w", "routed", "out", "res2", "y2"):
            assert torch.equal(got[n], want[n]), (i, n)


def test_training_step_of_gate_and_norm(nv):
    """Gradients through the gate, its losses and the norms in front, against float64 differentiation."""
    T, H, E, k = 150, 256, 24, 3
    g = torch.Generator(device=DEV).manual_seed(1)
    r = lambda *s: torch.randn(*s, device=DEV, generator=g)  # noqa: E731
    x, res, wg = r(T, H), r(T, H), r(E, H) * 0.1
    w_pre, w_post, gain = 1 + 0.1 * r(H), 1 + 0.1 * r(H), r(T, 1)
    d_w, d_loss = r(T, k), torch.tensor([0.5, 0.05], device=DEV)
    cu = torch.tensor([0, 70, 70, 149], dtype=torch.int32, device=DEV)
    res_out, y = nv.moe_block_norm(x, res, w_pre, w_post, gain, scale=0.7)
    logits = (y.double() @ wg.double().T).float()
    ids, w = nv.moe_gate_topk(logits, k, nv.SCORE_SQRT_SOFTPLUS)
    loss, counts, tokens = nv.moe_balance_loss(logits, ids, nv.SCORE_SQRT_SOFTPLUS, cu_seqlens=cu)
    d_logits = nv.moe_gate_backward(logits, ids, nv.SCORE_SQRT_SOFTPLUS, d_topk_w=d_w, d_loss=d_loss, counts=counts,
                                    tokens=tokens, cu_seqlens=cu)
    d_y = (d_logits.double() @ wg.double()).float()
    got = nv.moe_block_norm_backward(d_y, None, x, res_out, w_pre, w_post, gain, scale=0.7)
    leaves = [t.double().requires_grad_(True) for t in (x, res, w_pre, w_post, gain)]
    X, R, P, Q, A = leaves
    rms = lambda v: v / torch.sqrt(v.pow(2).mean(1, keepdim=True) + 1e-6)  # noqa: E731
    Y = rms(R + 0.7 * A * rms(X) * Q) * P
    s = torch.sqrt(torch.nn.functional.softplus(Y @ wg.double().T))
    sel = torch.gather(s, 1, ids.long())
    total = (sel / sel.sum(1, keepdim=True) * d_w.double()).sum()
    q = s / s.sum(1, keepdim=True)
    terms = [E * ((counts[i].double() / ((hi - lo) * k)) * q[lo:hi].mean(0)).sum() for i, (lo, hi) in
             ((0, (0, 70)), (2, (70, 149)))]
    z = torch.logsumexp(Y @ wg.double().T, 1)[:149].pow(2).mean()
    (total + 0.5 * (terms[0] + terms[1]) / 2 + 0.05 * z).backward()
    assert abs(loss[0].item() - (sum(terms) / 2).item()) <= 200 * EPS32 * abs(loss[0].item())
    for n, leaf in zip(("d_x", "d_residual", "d_w_pre", "d_w_post", "d_gate"), leaves):
        err = (got[n].double() - leaf.grad).abs().max().item()
        # a few hundred float32 roundings of terms at most ten times the largest gradient (sums that cancel)
        assert err <= 500 * EPS32 * 10 * leaf.grad.abs().max().item(), (n, err)


def test_two_streams_at_once(nv):
    """Different calls alternate on two streams without synchronization, each with its own workspace."""
    b = [Block(nv, 7), Block(nv, 8)]
    ins = [(q.r(200, q.H).bfloat16(), q.r(200, q.H).bfloat16(), torch.ones(200, dtype=torch.uint8, device=DEV)) for q in b]
    alone = [q.forward(nv, *i) for q, i in zip(b, ins)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(6):
        for n in (0, 1):
            with torch.cuda.stream(streams[n]):
                got[n].append(b[n].forward(nv, *ins[n]))
    torch.cuda.synchronize()
    for n in (0, 1):
        for d in got[n]:
            assert all(torch.equal(d[name], alone[n][name]) for name in ("ids", "w", "out", "res2", "y2"))


def test_offsets_past_32_bits(nv):
    """The last rows of tensors of more than 2^31 elements equal the same rows by themselves."""
    T, E = (1 << 31) // 1024 + 37, 1024
    x = torch.empty((T, E), dtype=torch.bfloat16, device=DEV)
    x[-64:] = torch.randn(64, E, device=DEV).bfloat16()
    x[:-64] = 0
    tail = x[-64:].clone()
    ids, w = nv.moe_gate_topk(x, 2)
    ids2, w2 = nv.moe_gate_topk(tail, 2)
    assert torch.equal(ids[-64:], ids2) and torch.equal(w[-64:], w2) and (ids[:-64] == torch.tensor([0, 1], device=DEV)).all()
    d = nv.moe_gate_backward(x, ids, renormalize=False, d_topk_w=torch.ones_like(w))
    d2 = nv.moe_gate_backward(tail, ids2, renormalize=False, d_topk_w=torch.ones_like(w2))
    assert torch.equal(d[-64:], d2)
    loss, counts, _ = nv.moe_balance_loss(x, ids)
    tail_counts = torch.bincount(ids2.flatten(), minlength=E)
    tail_counts[:2] += T - 64
    assert torch.equal(counts[0].long(), tail_counts)
    del x, d
    T, H = (1 << 31) // 7168 + 5, 7168
    x = torch.zeros((T, H), dtype=torch.bfloat16, device=DEV)
    x[-9:] = torch.randn(9, H, device=DEV).bfloat16()
    ones = torch.ones(H, device=DEV)
    r, y = nv.moe_block_norm(x, x, ones, ones)
    r2, y2 = nv.moe_block_norm(x[-9:].clone(), x[-9:].clone(), ones, ones)
    assert torch.equal(r[-9:], r2) and torch.equal(y[-9:], y2)
    g = nv.moe_block_norm_backward(y, None, x, r, ones, ones)
    g2 = nv.moe_block_norm_backward(y2, None, x[-9:].clone(), r2, ones, ones)
    assert torch.equal(g["d_x"][-9:], g2["d_x"]) and torch.equal(g["d_residual"][-9:], g2["d_residual"])
    del r, y, g
    q, s = nv.int8_quantize_rows(x)
    q2, s2 = nv.int8_quantize_rows(x[-9:].clone())
    assert torch.equal(q[-9:], q2) and torch.equal(s[-9:], s2)
    del x
    w_q, w_s = nv.int8_quantize_rows(torch.randn(64, H, device=DEV))
    out = nv.int8_gemm(q, s, w_q, w_s)
    assert torch.equal(out[-9:], nv.int8_gemm(q[-9:].clone(), s2, w_q, w_s))


def test_tensors_the_calls_refuse(nv):
    x = torch.randn(4, 16, device=DEV)
    ids, w = nv.moe_gate_topk(x, 2)
    q, s = nv.int8_quantize_rows(x)
    bad = [
        lambda: nv.moe_gate_topk(x.t(), 2), lambda: nv.moe_gate_topk(x.half(), 2), lambda: nv.moe_gate_topk(x[0], 2),
        lambda: nv.moe_gate_topk(x, 2, bias=torch.zeros(15, device=DEV)),
        lambda: nv.moe_gate_topk(x, 2, token_mask=torch.ones(4, device=DEV)),
        lambda: nv.moe_gate_topk(x, 2, topk_ids=torch.empty(7, dtype=torch.int32, device=DEV)),
        lambda: nv.moe_balance_loss(x, ids.long()), lambda: nv.moe_balance_loss(x, ids[:3]),
        lambda: nv.moe_balance_loss(x, ids, cu_seqlens=torch.zeros(1, dtype=torch.int32, device=DEV)),
        lambda: nv.moe_gate_backward(x, ids, d_loss=torch.ones(2, device=DEV)),
        lambda: nv.moe_gate_backward(x, ids, d_topk_w=torch.ones(4, 3, device=DEV)),
        lambda: nv.moe_block_norm(x, x.cpu()), lambda: nv.moe_block_norm(x, x[:3]),
        lambda: nv.moe_block_norm(x, x, torch.ones(15, device=DEV)),
        lambda: nv.moe_block_norm(x, x, gate=torch.ones(4, device=DEV)),
        lambda: nv.moe_block_norm_backward(x.bfloat16(), None, x, x, torch.ones(16, device=DEV)),
        lambda: nv.int8_quantize_rows(x.int()), lambda: nv.int8_gemm(q, s, q[:, :8].contiguous(), s),
        lambda: nv.int8_gemm(q, s[:3], q, s), lambda: nv.int8_gemm(q, s, q, s, add=x),
        lambda: nv.Int8FFNWeights(q, s, q, s),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    with pytest.raises(nv.NVFP4Error):
        nv.moe_gate_topk(x, 17)
    with pytest.raises(nv.NVFP4Error):
        nv.moe_gate_backward(x, ids)
    with pytest.raises(nv.NVFP4Error):
        nv.moe_balance_loss(x, ids, ws=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(nv.NVFP4Error):
        nv.int8_quantize_rows(torch.zeros(2, 24, device=DEV))
