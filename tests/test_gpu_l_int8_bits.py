"""The bits of 8-bit integer products: a token's outputs do not depend on the other tokens of the call, zeros' signs
included."""
import pytest
import torch

from _block_cases import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import nvfp4_quantized_moe_amd as nv
    return nv


@pytest.mark.parametrize("with_add", [False, True])
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("N,K", [(128, 64), (4096, 4096), (512, 8192), (528, 1040)])
def test_signs_of_zeros(nv, N, K, silu, with_add):
    """Up rows of zeros beside gates of both signs, and sums that meet scales too small for float32: the same bits in
    the kernels of few and of many tokens, undivided or in parts of K."""
    T = 700
    g = torch.Generator(device=DEV).manual_seed(N + K)
    a = torch.randint(-127, 128, (T, K), device=DEV, generator=g).to(torch.int8)
    b = torch.randint(-127, 128, (N, K), device=DEV, generator=g).to(torch.int8)
    b[N // 2::3] = 0
    a_s = torch.full((T,), 1e-3, device=DEV)
    a_s[::2] = 1e-30
    b_s = torch.full((N,), 1e-3, device=DEV)
    b_s[::2] = 1e-30
    n_out = N // 2 if silu else N
    add = torch.zeros((T, n_out), device=DEV).bfloat16()
    add[:, ::2] = -0.0
    epi = nv.EPI_SILU_MUL if silu else nv.EPI_BF16

    def bits(n):
        return nv.int8_gemm(a[:n], a_s[:n], b, b_s, epi, add=add[:n] if with_add else None).view(torch.int16)
    whole = bits(T)
    for n in (1, 16, 17, 40, 64, 130, 400):
        assert torch.equal(bits(n), whole[:n]), n
