"""silu(gate) * up of the MXFP4 products by itself: gates and ups whose sums are exact in float32, so that what is left
is the function's own error, in every kernel a product may take.

Only the first group of 128 elements holds anything: its first block of 32 makes the gates, its second the ups. Codes
times codes are multiples of 1/4 and 32 of them at most 1152, so the sums are exact in any order, and so are they times
the blocks' powers of two. e^-|g| by the hardware's power of two is off by its one step (2 half steps of float32, as the
reciprocal) and by the roundings of its argument, whose fraction is at most 1/2 (0.4); with the sum, the quotient and the
three products 8.4 half steps, whatever g is. Below g = -87.3 e^-|g| is subnormal, with an absolute half step of 2^-150,
down to -103.97, from where it is 0."""
import numpy as np
import pytest
import torch

import oracle.int8 as I8
import oracle.mxfp4 as MX
from _block_cases import DEV, EPS32, HALF_BF16, as_stored, to_dev

pytestmark = pytest.mark.gpu
SILU = 10 * EPS32


@pytest.fixture(scope="module")
def nv():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import nvfp4_quantized_moe_amd as nv
    return nv


def operands(M, N, K, up, seed):
    """Codes and scales of a product of gates around 2^0 to 2^8, half of them negative, and ups of size 2^up."""
    rng = np.random.default_rng(seed)
    a, b = np.zeros((M, K // 2), np.uint8), np.zeros((N, K // 2), np.uint8)
    a[:, :32], b[:N // 2, :16], b[N // 2:, 16:32] = (rng.integers(0, 256, s, dtype=np.uint8) for s in ((M, 32), (N // 2, 16), (N // 2, 16)))
    a_s, b_s = np.full((K // 128, M, 4), 127, np.uint8), np.full((K // 128, N, 4), 127, np.uint8)
    a_s[0, :, 0] = 127 + rng.integers(-2, 1, M)
    b_s[0, :N // 2, 0] = 127 + rng.integers(-3, 3, N // 2)
    b_s[0, N // 2:, 1] = 127 - 5 + up
    return a, a_s, b, b_s


def gate_up(a, a_s, b, b_s):
    A, B = (MX.dequantize(q[:, :64], s[:1]) for q, s in ((a, a_s), (b, b_s)))
    half = len(B) // 2
    return A @ B[:half].T, A @ B[half:].T


# a subtile of 16 tokens, two, the three tiles, parts of K and their join
SHAPES = [(5, 1040, 128), (32, 4096, 256), (200, 528, 128), (1500, 2064, 128), (4100, 4096, 128), (64, 4096, 16384)]


@pytest.mark.parametrize("up", [0, 10, 60])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_silu(nv, M, N, K, up):
    ops = operands(M, N, K, up, M + up)
    g, u = gate_up(*ops)
    for v in (g, u):
        assert np.array_equal(v.astype(np.float32), v)
    low = (g < -88) & (g > -100) & (u != 0)
    assert low.mean() > 0.001 and (g > 100).any() and (g < -110).any() and (np.abs(g) < 1).any()
    ref = I8.silu_mul(g, u)
    err = SILU * np.abs(ref) + (np.abs(g) + 2) * np.abs(u) * 2.0 ** -150 + 2.0 ** -150
    dev = [to_dev(v) for v in ops]
    got = nv.mxfp4_gemm(*dev, nv.EPI_SILU_MUL).double().cpu().numpy()
    worst = np.abs(got - ref) - err - HALF_BF16 * (np.abs(ref) + err) - 2.0 ** -134
    assert (worst <= 0).all(), (g[worst > 0][:5], u[worst > 0][:5], got[worst > 0][:5], ref[worst > 0][:5])
    # less the result's own BF16: what is left has the digits behind those, the sum is exact where it is small
    add = -as_stored(ref, "bf16")
    got = nv.mxfp4_gemm(*dev, nv.EPI_SILU_MUL, add=to_dev(add.astype(np.float32), torch.bfloat16)).double().cpu().numpy()
    left = ref + add
    worst = np.abs(got - left) - err - EPS32 * np.abs(left) - HALF_BF16 * (np.abs(left) + err) - 2.0 ** -134
    assert (worst <= 0).all(), (g[worst > 0][:5], float((worst / np.maximum(np.abs(ref), 1e-300)).max() / EPS32))
    # (half a step of BF16 of what is left is below the function's own error where little is left)
    assert M < 200 or (HALF_BF16 * np.abs(left) < EPS32 * np.abs(ref))[(g > -80) & (g < -40)].any()


def test_ends_of_the_range(nv):
    """The largest gates, infinite ones and NaN."""
    M = 3
    a, a_s, b, b_s = operands(M, 16, 128, 0, 1)
    a[:], b[:] = 0, 0
    a[:, 0], a[:, 16] = 0x02, 0x02                       # 1 in the first place of both blocks
    b[:8, 0], b[8:, 16] = 0x02, 0x02
    b[1::2][b[1::2] > 0] = 0x0A                        # and -1
    a_s[:], b_s[:] = 127, 127
    a_s[0, 1, 0] = 129                                   # 4 for the second token: 2^129 is infinite
    b_s[0, :8, 0] = [127, 127, 134, 134, 254, 254, 255, 127]
    g, u = gate_up(a, a_s, b, b_s)
    got = nv.mxfp4_gemm(*(to_dev(v) for v in (a, a_s, b, b_s)), nv.EPI_SILU_MUL).double().cpu().numpy()
    assert np.array_equal(g[:, 4], [2.0 ** 127, 2.0 ** 129, 2.0 ** 127])
    assert np.array_equal(got[:, 4], [2.0 ** 127, np.inf, 2.0 ** 127])
    assert (got[::2, 5] == 0).all() and (got[:, 3] == 0).all() and np.array_equal(got[:, 2], [128, 512, 128])
    assert np.isnan(got[:, 6]).all() and np.isfinite(got[:, [0, 1, 7]]).all()
