"""The 16-bit layer at its ends: no token, one more than the routing takes."""
import pytest
import torch

from tests.test_gpu_moe16 import layer, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("S", [0, 2])
@pytest.mark.parametrize("H,F", [(64, 96), (37, 61)])
def test_no_token(S, H, F):
    dt = torch.bfloat16
    lay = layer(dt, 5, 2, S, H, F)
    x, logits = rand((0, H), dt, 1), rand((0, 5), torch.float32, 2)
    assert lay.forward(x, logits).shape == (0, H)
    out, kept = lay.forward(x, logits, keep=True)
    g = lay.backward(torch.empty_like(out), kept, dw_dtype=torch.float32)
    assert g["dx"].shape == (0, H) and g["dlogits"].shape == (0, 5)
    for n, w in (("dw1", lay.w1), ("dw3", lay.w3), ("dw2", lay.w2)):
        assert g[n].shape == w.shape and not g[n].any()


def test_more_tokens_than_the_routing_takes():
    import extreme_quantized_moe_amd as m
    lay = layer(torch.bfloat16, 2, 1, 0, 8, 8)
    with pytest.raises(m._lib.MiloError, match="T="):
        lay.forward(rand((65537, 8), torch.bfloat16, 1), rand((65537, 2), torch.float32, 2))
