"""The MXFP4 calls refuse what they cannot compute, on the host, before any launch (CPU: the pointers are fake and
must never reach a kernel)."""
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


def test_padded(nv):
    assert [nv.mxfp4_padded(n) for n in (0, 1, 128, 129, 262144)] == [0, 128, 128, 256, 262144]
    for n in (-1, 262145):
        with pytest.raises(ValueError):
            nv.mxfp4_padded(n)


def test_quantize(nv):
    def call(x=P, dt=0, M=4, K=64, rule=0, q=P, s=P, qt=None, st=None):
        return nv._mx_quantize(x, dt, M, K, rule, q, s, qt, st, None)
    for bad in (dict(M=-1), dict(K=0), dict(K=12), dict(K=262152), dict(M=64 * 65535 + 1),
                dict(M=262145, qt=P, st=P)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(dt=2), dict(rule=2), dict(rule=-1)):
        assert call(**bad) == ARG, bad
    for bad in (dict(x=None), dict(q=None), dict(s=None), dict(q=None, s=None), dict(qt=P), dict(st=P)):
        assert call(**bad) == NULL, bad
    for bad in (dict(x=ODD), dict(q=ODD), dict(s=ODD), dict(qt=ODD, st=P), dict(qt=P, st=ODD)):
        assert call(**bad) == ALIGN, bad
    assert call(M=0, x=None) == 0


def test_dequantize(nv):
    def call(q=P, s=P, R=4, K=128, cols=100, dt=0, out=P):
        return nv._mx_dequantize(q, s, R, K, cols, dt, out, None)
    for bad in (dict(R=-1), dict(K=96), dict(K=262272), dict(cols=-1), dict(cols=129), dict(R=64 * 65535 + 1)):
        assert call(**bad) == SHAPE, bad
    assert call(dt=3) == ARG
    for bad in ("q", "s", "out"):
        assert call(**{bad: None}) == NULL and call(**{bad: ODD}) == ALIGN, bad
    assert call(R=0, q=None) == 0 and call(cols=0, out=None) == 0


def test_gemm(nv):
    def call(a=P, a_s=P, b=P, b_s=P, M=4, N=64, K=128, epi=0, add=None, dt=0, d=P, ws=None, n=0):
        return nv._mx_gemm(a, a_s, b, b_s, M, N, K, epi, add, dt, d, ws, n, None)
    for bad in (dict(M=-1), dict(N=0), dict(N=12), dict(N=24, epi=1), dict(K=64), dict(K=-128), dict(K=262272),
                dict(M=64 * 65535 + 1), dict(N=(1 << 27) - 8), dict(M=1 << 20, K=1 << 16), dict(N=1 << 20, K=1 << 16)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(epi=2), dict(epi=-1), dict(dt=2), dict(epi=1, dt=1)):
        assert call(**bad) == ARG, bad
    for bad in ("a", "a_s", "b", "b_s", "d"):
        assert call(**{bad: None}) == NULL and call(**{bad: ODD}) == ALIGN, bad
    assert call(add=ODD) == ALIGN and call(M=0, a=None) == 0 and call(K=0, d=None) == NULL
    assert call(M=64 * 65535, N=1 << 26, K=128) == SHAPE
    parts = nv.mxfp4_gemm_ws_bytes(64, 4096, 16384)
    assert parts > 0 and nv.mxfp4_gemm_ws_bytes(8192, 4096, 16384) == 0 and nv.mxfp4_gemm_ws_bytes(64, 12, 16384) == 0
    assert nv.mxfp4_gemm_ws_bytes(0, 4096, 16384) == 0
    assert call(M=64, N=4096, K=16384) == NULL and call(M=64, N=4096, K=16384, ws=ODD, n=parts) == ALIGN
    assert call(M=64, N=4096, K=16384, ws=P, n=parts - 1) == WORKSPACE


def test_calls_refuse_what_is_no_gpu_tensor(nv):
    import torch
    x, q, s = torch.zeros(4, 128), torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(1, 4, 4, dtype=torch.uint8)
    for i, call in enumerate((lambda: nv.mxfp4_quantize(x), lambda: nv.mxfp4_quantize(x.half()),
                              lambda: nv.mxfp4_dequantize(q, s), lambda: nv.mxfp4_dequantize(q, s, torch.float16),
                              lambda: nv.mxfp4_gemm(q, s, q, s), lambda: nv.mxfp4_gemm(q, None, q, s),
                              lambda: nv.mxfp4_gemm(q, s, q, s, dtype=torch.float64))):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
