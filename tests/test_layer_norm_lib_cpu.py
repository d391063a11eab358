"""The layer norm refuses what it cannot compute, on the host, before any launch (CPU: the pointers are fake and must
never reach a kernel)."""
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


def test_forward(nv):
    def call(x=P, xt=0, r=P, rt=0, T=4, H=64, w=P, b=P, scale=0.5, out=P, y=P, rule=0, q=None, s=None):
        return nv._layer_norm(x, xt, r, rt, T, H, w, b, scale, 1e-5, out, y, rule, q, s, None)
    for bad in (dict(T=-1), dict(H=0), dict(H=60), dict(H=16392)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(xt=2), dict(rt=-1), dict(rule=2, q=P, s=P), dict(r=None, out=None), dict(r=None, scale=1.0),
                dict(r=None, out=None, scale=1.0, rt=1)):
        assert call(**bad) == ARG, bad
    for bad in (dict(x=None), dict(out=None), dict(y=None), dict(q=P), dict(s=P)):
        assert call(**bad) == NULL, bad
    for bad in ("x", "r", "w", "b", "out", "y"):
        assert call(**{bad: ODD}) == ALIGN, bad
    assert call(q=ODD, s=P) == ALIGN and call(q=P, s=ODD) == ALIGN
    assert call(T=0, x=None, r=None, out=None, y=None) == 0


def test_backward(nv):
    need = nv.moe_layer_norm_backward_ws_bytes(4, 64)
    assert need > 0 and nv.moe_layer_norm_backward_ws_bytes(4, 60) == 0 and nv.moe_layer_norm_backward_ws_bytes(-1, 64) == 0

    def call(dy=P, xt=0, dro=P, r=P, rt=0, T=4, H=64, w=P, scale=0.5, dx=P, dr=P, dw=P, db=P, ws=P, n=need):
        return nv._layer_norm_backward(dy, xt, dro, r, rt, T, H, w, scale, 1e-5, dx, dr, dw, db, ws, n, None)
    for bad in (dict(T=-1), dict(H=4), dict(H=16392)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(xt=3), dict(rt=3), dict(dr=None), dict(dr=None, scale=1.0, rt=1)):
        assert call(**bad) == ARG, bad
    for bad in ("dy", "r", "dx", "ws"):
        assert call(**{bad: None}) == NULL, bad
    for bad in ("dy", "dro", "r", "w", "dx", "dr", "dw", "db", "ws"):
        assert call(**{bad: ODD}) == ALIGN, bad
    assert call(n=need - 1) == WORKSPACE
