"""The largest sizes that the operators around the expert FFN take: past them they refuse on the host (CPU: the
pointers are fake and must never reach a kernel)."""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "nvfp4_quantized_moe_amd", "libnvfp4moe.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="library not built (run build())")

SHAPE = 2
P = ctypes.c_void_p(4096)


def test_columns_past_a_grid():
    """The kernel of few tokens runs 512 threads for 16 columns; a launch holds fewer than 2^32."""
    import nvfp4_quantized_moe_amd as nv
    for n in range((1 << 27) - 8, (1 << 27) + 8, 8):
        assert nv._int8_gemm(P, P, P, P, 1, n, 16, 0, None, P, None, 0, None) == SHAPE
    assert nv.int8_gemm_ws_bytes(1, (1 << 27) - 8, 16) == 0
