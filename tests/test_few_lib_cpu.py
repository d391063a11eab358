"""The layer for a few tokens refuses what it cannot compute, on the host, before any launch (CPU: the pointers are
fake and must never reach a kernel); its oracle on a worked layer."""
import ctypes
import os

import numpy as np
import pytest

import oracle.few as F

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "nvfp4_quantized_moe_amd", "libnvfp4moe.so")

NULL, SHAPE, ALIGN, WORKSPACE, ARG = 1, 2, 3, 4, 6
built = pytest.mark.skipif(not os.path.exists(LIB), reason="library not built (run build())")


@built
def test_refusals():
    import nvfp4_quantized_moe_amd as nv
    assert nv.nvfp4_moe_few_max_tokens() == 64
    need = nv.nvfp4_moe_few_ws_bytes(4, 2, 256, 128, 8)
    assert need >= 4 * 2 * 128 * 2
    for bad in ((65, 2, 256, 128, 8), (-1, 2, 256, 128, 8), (4, 0, 256, 128, 8), (4, 65, 256, 128, 8),
                (4, 2, 192, 128, 8), (4, 2, 256, 64, 8), (4, 2, 256, 128, 0), (4, 2, 256, 128, 4097),
                (4, 2, 65536, 65536, 8)):
        assert nv.nvfp4_moe_few_ws_bytes(*bad) == 0, bad

    def call(w=True, w1=4096, gs1=4096, w2=4096, gs2=4096, L=8, H=256, I=128, dual=0, x=4096, T=4, ids=4096, tw=4096, k=2,
             add=None, out=4096, ws=4096, n=need):
        s = nv._Weights(L, H, I, w1, gs1, w2, gs2, dual)
        return nv._few(ctypes.byref(s) if w else None, x, T, ids, tw, k, 0, add, out, ws, n, None)
    for bad in (dict(T=65), dict(T=-1), dict(k=0), dict(k=65), dict(H=192), dict(I=64), dict(L=0), dict(L=4097),
                dict(H=0), dict(H=65536, I=65536)):
        assert call(**bad) == SHAPE, bad
    assert call(dual=2) == ARG and call(w=False) == NULL
    for bad in ("w1", "gs1", "w2", "gs2", "x", "ids", "tw", "out", "ws"):
        assert call(**{bad: None}) == NULL, bad
    for bad in ("w1", "w2", "x", "add", "out", "ws"):
        assert call(**{bad: 4100}) == ALIGN, bad
    assert call(n=need - 1) == WORKSPACE and call(T=0, x=None, ids=None, tw=None, out=None, ws=None) == 0


def test_worked_layer():
    """One hidden unit: out = w (w2 bf16(silu(g) u)), added to what there is, experts of other ranks left out."""
    w1 = np.array([[[2.0], [3.0]], [[-1.0], [0.5]]])      # [L, 2I, H] with I = H = 1
    w2 = np.array([[[4.0]], [[8.0]]])
    x = np.array([[1.0], [2.0]])
    ids, w = np.array([[5, 6], [7, 5]]), np.array([[0.5, 0.25], [1.0, 2.0]], np.float32)
    out, size = F.forward(x, ids, w, 5, w1, w2, add=np.array([[1.0], [-1.0]]))

    def h(g, u):
        v = g / (1 + np.exp(-g)) * u
        return np.round(v * 2 ** (7 - np.floor(np.log2(abs(v))))) / 2 ** (7 - np.floor(np.log2(abs(v))))
    assert out[0, 0] == 1 + 0.5 * 4 * h(2.0, 3.0) + 0.25 * 8 * h(-1.0, 0.5)
    assert out[1, 0] == -1 + 2 * 4 * h(4.0, 6.0)          # expert 7 lives elsewhere
    assert size[1, 0] == 1 + 2 * 4 * h(4.0, 6.0)
