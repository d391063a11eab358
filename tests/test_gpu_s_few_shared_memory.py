"""The layer for a few tokens around the sizes at which the down products' tokens no longer fit LDS beside their sums:
the last number of choices that does, and the next one."""
import pytest
import torch

from _block_cases import DEV, to_dev
from test_gpu_o_few import check, choices, layer, nv  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["plain", "twice"])
@pytest.mark.parametrize("T,k", [(60, 32), (60, 33), (61, 28), (61, 29), (61, 30), (62, 25), (62, 26), (63, 21), (63, 22),
                                 (63, 23), (64, 18), (64, 19)])
def test_layer(nv, T, k, kind):  # noqa: F811
    E, L, start, H, I = 240, 160, 20, 256, 128   # experts of about six tokens: some above eight
    weights, w1, w2, g = layer(nv, L, H, I, False, T + k)
    ids, w = choices(kind, T, k, E, start, L, T)
    x, add = (torch.randn(T, H, device=DEV, generator=g).bfloat16() for _ in range(2))
    ws = torch.full((nv.nvfp4_moe_few_ws_bytes(T, k, H, I, L),), 0xFF, dtype=torch.uint8, device=DEV)
    out = nv.nvfp4_moe_forward_few(weights, x, to_dev(ids), to_dev(w), start, add=add, ws=ws)
    check(x, ids, w, start, weights, w1, w2, ws[:T * k * I * 2].view(torch.bfloat16).view(T, k, I), out, add)
    assert torch.equal(nv.nvfp4_moe_forward_few(weights, x, to_dev(ids), to_dev(w), start, add=add), out)
