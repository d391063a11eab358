"""What limits a call of the MXFP4 inverse is the columns asked for, not those behind them (CPU: the call with a null
pointer gets past the sizes' checks, and no kernel is reached)."""
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "nvfp4_quantized_moe_amd", "libnvfp4moe.so")
NULL, SHAPE = 1, 2
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="library not built (run build())")


@pytest.mark.parametrize("R,K,cols,dt,want", [
    (64 * 65535, 262144, 128, 0, NULL), (64 * 65535, 262144, 256, 1, NULL), (64 * 65535, 65536, 1, 1, NULL),
    (64 * 65535, 65536, 65536, 0, NULL), (64 * 65535, 65664, 65664, 0, SHAPE), (64 * 65535, 32896, 32896, 1, SHAPE)])
def test_dequantize(R, K, cols, dt, want):
    import nvfp4_quantized_moe_amd as nv
    assert nv._mx_dequantize(None, None, R, K, cols, dt, None, None) == want
