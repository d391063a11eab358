"""The operators around the expert FFN refuse what they cannot compute, on the host, before any launch (CPU: the
pointers are fake and must never reach a kernel)."""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "nvfp4_quantized_moe_amd", "libnvfp4moe.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="library not built (run build())")

NULL, SHAPE, ALIGN, WORKSPACE, ARG = 1, 2, 3, 4, 6
P, ODD = ctypes.c_void_p(4096), ctypes.c_void_p(4100)


@pytest.fixture(scope="module")
def nv():
    import nvfp4_quantized_moe_amd as nv
    return nv


def test_gate_topk(nv):
    def call(logits=P, dtype=1, bias=None, mask=None, T=4, E=64, k=8, score=0, groups=1, top=1, renorm=1, ids=P, w=P):
        return nv._gate_topk(logits, dtype, bias, mask, T, E, k, score, groups, top, renorm, 1.0, ids, w, None)
    for bad in (dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=65, E=128), dict(k=9, E=8), dict(T=1 << 28),
                dict(groups=0), dict(groups=3), dict(groups=128, E=128), dict(groups=8, top=9), dict(groups=8, top=0),
                dict(groups=16, top=1, k=5)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(dtype=2), dict(score=3), dict(score=-1), dict(renorm=2)):
        assert call(**bad) == ARG, bad
    for bad in (dict(logits=None), dict(ids=None), dict(w=None)):
        assert call(**bad) == NULL, bad
    for bad in (dict(logits=ODD), dict(ids=ODD), dict(w=ODD), dict(bias=ODD), dict(mask=ODD)):
        assert call(**bad) == ALIGN, bad
    assert call(T=0, logits=None, ids=None, w=None) == 0


def test_balance_loss(nv):
    need = nv.moe_balance_loss_ws_bytes(4, 64, 2)
    assert need > 0 and nv.moe_balance_loss_ws_bytes(4, 64, 0) == 0 and nv.moe_balance_loss_ws_bytes(4, 2000, 1) == 0

    def call(logits=P, dtype=1, ids=P, mask=None, cu=P, B=2, T=4, E=64, k=8, score=0, loss=P, counts=P, tokens=P, ws=P,
             n=need):
        return nv._balance(logits, dtype, ids, mask, cu, B, T, E, k, score, loss, counts, tokens, ws, n, None)
    for bad in (dict(T=-1), dict(E=1025), dict(k=65), dict(B=0), dict(B=65536), dict(cu=None)):
        assert call(**bad) == SHAPE, bad
    assert call(dtype=9) == ARG and call(score=4) == ARG
    for bad in ("logits", "ids", "loss", "counts", "tokens", "ws"):
        assert call(**{bad: None}) == NULL, bad
    for bad in ("logits", "ids", "mask", "cu", "loss", "counts", "tokens", "ws"):
        assert call(**{bad: ODD}) == ALIGN, bad
    assert call(n=need - 1) == WORKSPACE


def test_gate_backward(nv):
    def call(logits=P, dtype=1, ids=P, mask=None, T=4, E=64, k=8, score=0, renorm=1, d_w=P, d_loss=P, counts=P, tokens=P,
             cu=P, B=2, out=P):
        return nv._gate_backward(logits, dtype, ids, mask, T, E, k, score, renorm, 1.0, d_w, d_loss, counts, tokens, cu,
                                 B, out, None)
    for bad in (dict(T=-1), dict(E=0), dict(k=65), dict(B=0), dict(cu=None)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(dtype=5), dict(score=7), dict(renorm=3)):
        assert call(**bad) == ARG, bad
    for bad in (dict(logits=None), dict(ids=None), dict(d_w=None, d_loss=None), dict(counts=None), dict(tokens=None),
                dict(out=None)):
        assert call(**bad) == NULL, bad
    for bad in ("logits", "ids", "mask", "d_w", "d_loss", "counts", "tokens", "cu", "out"):
        assert call(**{bad: ODD}) == ALIGN, bad
    assert call(T=0) == 0


def test_binding_refuses_tensors_on_the_host(nv):
    import torch
    x = torch.zeros(4, 16)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: nv.moe_gate_topk(x, 2), lambda: nv.moe_balance_loss(x, ids),
                 lambda: nv.moe_gate_backward(x, ids, d_topk_w=torch.zeros(4, 2)),
                 lambda: nv.moe_gate_topk(x.double(), 2)):
        with pytest.raises(ValueError):
            call()


def test_block_norm(nv):
    def call(x=P, xt=0, r=P, rt=0, T=4, H=64, w_pre=P, w_post=P, gate=P, mode=1, out=P, y=P, gs=None, q=None, sf=None):
        return nv._block_norm(x, xt, r, rt, T, H, w_pre, w_post, gate, mode, 1.0, 1e-6, out, y, gs, q, sf, None)
    for bad in (dict(T=-1), dict(H=0), dict(H=60), dict(H=16392), dict(H=40, gs=P, q=P, sf=P)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(xt=2), dict(rt=-1), dict(mode=3), dict(xt=1, gs=P, q=P, sf=P)):
        assert call(**bad) == ARG, bad
    for bad in (dict(x=None), dict(out=None), dict(y=None), dict(gate=None), dict(gs=P), dict(gs=P, q=P),
                dict(gs=P, q=P, sf=P, w_pre=None)):
        assert call(**bad) == NULL, bad
    for bad in ("x", "r", "w_pre", "w_post", "gate", "out", "y"):
        assert call(**{bad: ODD}) == ALIGN, bad
    assert call(gs=ODD, q=P, sf=P) == ALIGN and call(gs=P, q=ODD, sf=P) == ALIGN and call(gs=P, q=P, sf=ODD) == ALIGN
    assert call(T=0, x=None, r=None, out=None, y=None) == 0


def test_block_norm_backward(nv):
    need = nv.moe_block_norm_backward_ws_bytes(4, 64)
    assert need > 0 and nv.moe_block_norm_backward_ws_bytes(4, 60) == 0

    def call(d_y=P, d_r=P, x=P, xt=0, r=P, rt=0, T=4, H=64, w_pre=P, w_post=P, gate=P, mode=1, dx=P, dr=P, a=P, b=P, c=P,
             ws=P, n=need):
        return nv._block_norm_backward(d_y, d_r, x, xt, r, rt, T, H, w_pre, w_post, gate, mode, 1.0, 1e-6, dx, dr, a, b,
                                       c, ws, n, None)
    for bad in (dict(T=-1), dict(H=4), dict(H=16392)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(xt=3), dict(rt=3), dict(mode=5)):
        assert call(**bad) == ARG, bad
    for bad in (dict(d_y=None), dict(x=None), dict(r=None), dict(dx=None), dict(dr=None), dict(a=None), dict(b=None),
                dict(c=None), dict(gate=None), dict(ws=None), dict(w_pre=None, d_r=None)):
        assert call(**bad) == NULL, bad
    for bad in ("d_y", "d_r", "x", "r", "w_pre", "w_post", "gate", "dx", "dr", "a", "b", "c", "ws"):
        assert call(**{bad: ODD}) == ALIGN, bad
    assert call(n=need - 1) == WORKSPACE


def test_int8(nv):
    def rows(x=P, xt=0, M=4, K=64, q=P, s=P):
        return nv._int8_rows(x, xt, M, K, q, s, None)
    for bad in (dict(M=-1), dict(K=0), dict(K=24), dict(K=65552)):
        assert rows(**bad) == SHAPE, bad
    assert rows(xt=2) == ARG
    for bad in ("x", "q", "s"):
        assert rows(**{bad: None}) == NULL and rows(**{bad: ODD}) == ALIGN, bad
    assert rows(M=0, x=None) == 0

    def gemm(a=P, a_s=P, b=P, b_s=P, M=4, N=64, K=64, epi=0, add=None, d=P, ws=None, n=0):
        return nv._int8_gemm(a, a_s, b, b_s, M, N, K, epi, add, d, ws, n, None)
    for bad in (dict(M=-1), dict(N=0), dict(N=12), dict(N=24, epi=1), dict(K=8), dict(K=40), dict(K=65552),
                dict(M=64 * 65535 + 1)):
        assert gemm(**bad) == SHAPE, bad
    assert gemm(epi=2) == ARG and gemm(epi=-1) == ARG
    for bad in ("a", "a_s", "b", "b_s", "d"):
        assert gemm(**{bad: None}) == NULL and gemm(**{bad: ODD}) == ALIGN, bad
    assert gemm(add=ODD) == ALIGN and gemm(M=0, a=None) == 0
    parts = nv.int8_gemm_ws_bytes(64, 512, 8192)
    assert parts > 0 and nv.int8_gemm_ws_bytes(8192, 4096, 8192) == 0 and nv.int8_gemm_ws_bytes(64, 12, 8192) == 0
    assert gemm(M=64, N=512, K=8192) == NULL and gemm(M=64, N=512, K=8192, ws=ODD, n=parts) == ALIGN
    assert gemm(M=64, N=512, K=8192, ws=P, n=parts - 1) == WORKSPACE

    need = nv.int8_ffn_ws_bytes(4, 64, 32)
    assert need > 0 and nv.int8_ffn_ws_bytes(4, 64, 24) == 0

    def ffn(w1=P, s1=P, w2=P, s2=P, x=P, T=4, H=64, I=32, add=None, out=P, ws=P, n=need):
        return nv._int8_ffn(w1, s1, w2, s2, x, T, H, I, add, out, ws, n, None)
    for bad in (dict(T=-1), dict(H=40), dict(I=24), dict(H=0), dict(I=65552), dict(T=64 * 65535 + 1)):
        assert ffn(**bad) == SHAPE, bad
    for bad in ("w1", "s1", "w2", "s2", "x", "out", "ws"):
        assert ffn(**{bad: None}) == NULL and ffn(**{bad: ODD}) == ALIGN, bad
    assert ffn(add=ODD) == ALIGN and ffn(n=need - 1) == WORKSPACE and ffn(T=0, x=None, out=None) == 0


def test_sizes_past_a_grid(nv):
    assert nv._gate_topk(P, 1, None, None, 1 << 26, 4, 1, 0, 1, 1, 1, 1.0, P, P, None) == SHAPE
    assert nv._balance(P, 1, P, None, None, 1, 1 << 26, 4, 1, 0, P, P, P, P, 1 << 40, None) == SHAPE
    assert nv._gate_backward(P, 1, P, None, 1 << 26, 4, 1, 0, 1, 1.0, P, None, None, None, None, 1, P, None) == SHAPE
    assert nv._int8_rows(P, 0, 64 * 65535 + 1, 64, P, P, None) == SHAPE
    assert nv._int8_gemm(P, P, P, P, 1, 1 << 27, 16, 0, None, P, None, 0, None) == SHAPE
    assert nv._int8_gemm(P, P, P, P, 64 * 65535, 1 << 26, 16, 0, None, P, None, 0, None) == SHAPE


def test_calls_refuse_what_is_no_gpu_tensor(nv):
    """The Python calls look at their tensors first: nothing here needs a device."""
    import torch
    x, ids = torch.zeros(4, 16), torch.zeros(4, 2, dtype=torch.int32)
    q, s = torch.zeros(4, 16, dtype=torch.int8), torch.zeros(4)
    calls = [lambda: nv.moe_gate_topk(x, 2), lambda: nv.moe_balance_loss(x, ids),
             lambda: nv.moe_gate_backward(x, ids, d_topk_w=x), lambda: nv.moe_block_norm(x, x),
             lambda: nv.moe_block_norm_backward(None, x, x, x), lambda: nv.int8_quantize_rows(x),
             lambda: nv.int8_gemm(q, s, q, s), lambda: nv.prepare_int8_weights(x, x, x.t()),
             lambda: nv.moe_gate_topk(x.half(), 2), lambda: nv.int8_gemm(q, None, q, s), lambda: nv.int8_gemm(None, s, q, s)]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    for call in (lambda: nv.moe_gate_topk([[1.0]], 1), lambda: nv.moe_block_norm("x", x), lambda: nv._native.gemm(q)):
        with pytest.raises(TypeError):
            call()
