"""Outputs handed to the 16-bit operators that share memory with an input are
refused; the gate operand and the residual may be the output itself."""
import pytest
import torch

import extreme_quantized_moe_amd as m
from extreme_quantized_moe_amd.moe16 import _apart


def test_shared_memory_is_refused():
    buf = torch.zeros(64, dtype=torch.float16)
    a, b = buf[:16].view(2, 8), buf[16:32].view(2, 8)
    _apart(a, b, None)
    _apart(b, a, buf[32:])
    _apart(a, b, same=(a, None))
    _apart(a[:0], a)                                    # no memory at all
    for bad in (lambda: _apart(a, a), lambda: _apart(a, b, buf), lambda: _apart(a, a, same=(a,)),
                lambda: _apart(buf[8:24], b),
                lambda: _apart(a, same=(buf[1:17].view(2, 8),)),            # the same size, a row off
                lambda: _apart(a.view(-1).view(torch.float32), same=(a,))):  # of another type
        with pytest.raises(ValueError, match="shares memory"):
            bad()


@pytest.mark.gpu
def test_operators_refuse_an_output_over_an_input():
    def r(*shape):
        return torch.randn(shape, device="cuda").bfloat16()
    x, w, y = r(4, 64), r(64, 64), r(8, 64)
    pos = torch.arange(8, dtype=torch.int32, device="cuda")
    big = r(12, 64)
    for bad in (lambda: m.moe_linear(x, w, out=x), lambda: m.moe_linear(x, w, out=w[:4]),
                lambda: m.moe_linear(x, w, mul=big[:4], out=big[1:5]),
                lambda: m.moe_permute(big[:4], pos, 2, out=big[2:10]),
                lambda: m.moe_unpermute(big[:8], pos, 2, out=big[:4]),
                lambda: m.moe_unpermute_grad(x, y, pos, 2, out=y),
                lambda: m.moe_unpermute_grad(big[:4], y, pos, 2, out=big[:8])):
        with pytest.raises(ValueError, match="shares memory"):
            bad()
    res = r(4, 64)
    want = m.moe_linear(x, w, residual=res)
    assert torch.equal(m.moe_linear(x, w, residual=res, out=res), want)
