"""The Python calls of the operators around the expert FFN look at every tensor of every call."""
import pytest
import torch

from _block_cases import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import nvfp4_quantized_moe_amd as nv
    return nv


def test_weights_set_after_they_were_made(nv):
    """Attributes of Int8FFNWeights are a user's to set; the call refuses what the kernels could not read."""
    H, I = 64, 32

    def made():
        return nv.prepare_int8_weights(torch.randn(I, H, device=DEV), torch.randn(I, H, device=DEV),
                                       torch.randn(H, I, device=DEV))
    x = torch.randn(5, H, device=DEV).bfloat16()
    good = made()
    for name in ("w1_q", "w1_scale", "w2_q", "w2_scale"):
        t = getattr(good, name)
        for bad in (t.cpu(), t[:-1].contiguous(), t.to(torch.int32), None):
            w = made()
            setattr(w, name, bad)
            with pytest.raises(ValueError):
                nv.int8_ffn_forward(w, x)
    other, w = made(), made()
    for name in ("w1_q", "w1_scale", "w2_q", "w2_scale"):
        setattr(w, name, getattr(other, name))
    assert torch.equal(nv.int8_ffn_forward(w, x), nv.int8_ffn_forward(other, x))
