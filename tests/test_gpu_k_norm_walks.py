"""The block norms where a workgroup walks several rows, and where several row groups add their column sums: the
checks and tolerances of test_gpu_g_norm.py at sizes with more than one turn.

Forward, 256 CUs hold up to 16 waves each: T above 256 * (16 / waves of a row). Backward, a workgroup has 768 threads
(512 with two chunks per thread or more) in row groups of whole waves, and there are 256 workgroups.
"""
import pytest
import torch

import test_gpu_g_norm as norm
from test_gpu_g_norm import case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import nvfp4_quantized_moe_amd as nv
    return nv


def name(c):
    return f"T{c['T']}-H{c['H']}-{c['x']}-{c['res']}-{c['gate']}"


FORWARD = [
    case(9001, 64, gate="token"), case(9000, 128, "f32", "f32"), case(2700, 1032, "bf16", "f32"),
    case(1100, 4096, gate=None, post=False), case(1100, 7168), case(1100, 7168, pre=False, gate="token"),
    case(800, 8200, "f32", "bf16", "token"), case(600, 16384, "bf16", "bf16"),
    case(9001, 40, pre=False, post=False, gate=None),
]


@pytest.mark.parametrize("c", FORWARD, ids=map(name, FORWARD))
def test_forward_of_walked_rows(nv, c):
    norm.test_forward(nv, c)


BACKWARD = [
    # twelve row groups, the last turn partly filled
    case(7000, 64, "f32", "f32"), case(7001, 128), case(7001, 128, gate="token", post=False), case(6500, 512, "bf16", "f32"),
    # fewer rows: 5, 7, 8, 9, 10 and 11 row groups, one turn
    case(1200, 64), case(1700, 64, "f32", "bf16"), case(2000, 72), case(2200, 64, gate="token"), case(2400, 80, "bf16", "f32"),
    case(2700, 64, gate=None),
    # six, four, three and two groups over several turns
    case(3500, 776), case(2500, 1032, gate="token"), case(1800, 2048, "f32", "f32"), case(1100, 2888, "bf16", "f32", "token"),
    # two chunks per thread in two groups and in one, four chunks (no weights in registers)
    case(1100, 4096), case(1101, 3080, "f32", "bf16", "token"), case(600, 7168), case(601, 7168, pre=False),
    case(530, 8200, "bf16", "f32"), case(520, 16384, gate="token"),
]


@pytest.mark.parametrize("c", BACKWARD, ids=map(name, BACKWARD))
def test_backward_of_walked_rows(nv, c):
    norm.test_backward(nv, c, True)


@pytest.mark.parametrize("c", [case(7001, 128), case(600, 7168, gate="token")], ids=name)
def test_backward_of_walked_rows_without_a_residual_gradient(nv, c):
    norm.test_backward(nv, c, False)


@pytest.mark.parametrize("T,H", [(1300, 7168), (9001, 96), (900, 8224)])
def test_nvfp4_output_of_walked_rows(nv, T, H):
    norm.test_nvfp4_output_equals_the_static_quantizer(nv, T, H, "bf16", 1.0)


@pytest.mark.parametrize("T,H", [(7001, 128), (1101, 4096), (600, 7168), (601, 8200)])
def test_in_place_over_several_turns(nv, T, H):
    """Gradients over their inputs, and the update over the residual and x: as with buffers apart."""
    p, _ = norm.inputs(case(T, H), 6)
    bf16 = lambda a: norm.to_dev(a.astype("float32"), torch.bfloat16)  # noqa: E731
    x, r, w, wp, g = bf16(p["x"]), bf16(p["residual"]), *(norm.f32_dev(p[n]) for n in ("w_pre", "w_post", "gate"))
    r1, y1 = nv.moe_block_norm(x, r, w, wp, g)
    d_y, d_r = torch.randn_like(x), torch.randn_like(r)
    apart = nv.moe_block_norm_backward(d_y, d_r, x, r1, w, wp, g)
    over = nv.moe_block_norm_backward(d_y, d_r, x, r1, w, wp, g, d_x=d_y, d_residual=d_r)
    assert all(torch.equal(apart[n], over[n]) for n in apart)
    nv.moe_block_norm(x, r, w, wp, g, residual_out=r, y=x)
    assert torch.equal(r, r1) and torch.equal(x, y1)
