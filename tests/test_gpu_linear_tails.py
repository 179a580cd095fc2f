"""Activations and their slopes in float32, relative to themselves, out to where
the exponential flushes.

Bounds, in roundings U = 2^-24 of the value.  exp2's argument is -a log2(e)
rounded once, with a constant that is off by 0.22 U: the result is off by up to
1.22 a U, and by 2 U of the instruction; reciprocal, products and the fit of
erfcx (2.2 U) add up to 10 U (SiLU) and 22 U (GELU).  a = |v| for SiLU, v^2 / 2
for GELU (v^2 is kept to twice the precision).  GELU_TANH's a = 2 c |v + 0.044715
v^3| takes two products, a sum, another product and two rounded constants: 5.2 U
of a before the 1.22.  The slopes are sums of two terms, each with the error of
its factors, 1 - g with another 4 U of 1."""
import math

import pytest
import torch

from tests.moe16_reference import F64, U32, act, act_slope, check, lost_slope, lost_value

pytestmark = pytest.mark.gpu
C2 = 2 * math.sqrt(2 / math.pi)
FAR = {"silu": 87.0, "gelu": 13.1, "gelu_tanh": 9.9}       # exp(-a) reaches 2^-126


def grid(name, dt):
    """256 x 64 arguments over the whole range, half of them in [-4, 4]."""
    g = torch.Generator().manual_seed(5)
    v = (torch.rand((256, 64), generator=g, dtype=F64) * 2 - 1) * FAR[name]
    v[:, 32:] = torch.rand((256, 32), generator=g, dtype=F64) * 8 - 4
    return v.to(dt).cuda()


def parts(name, v):
    """(a, roundings of the exponential's side, g) of the value v g."""
    if name == "silu":
        return v.abs(), 1.25 * v.abs() + 10, torch.sigmoid(v)
    if name == "gelu":
        return v * v / 2, 1.25 * v * v / 2 + 22, 0.5 * torch.erfc(-v / math.sqrt(2))
    a = C2 * (v + 0.044715 * v ** 3).abs()
    return a, 6.5 * a + 12, torch.sigmoid(C2 * (v + 0.044715 * v ** 3))


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
def test_values(name, dt):
    import extreme_quantized_moe_amd as m
    x = grid(name, dt)
    eye = torch.eye(64, dtype=dt, device="cuda")
    v = x.to(F64)
    want = act(name, v)
    _, r, _ = parts(name, v)
    for rows in (slice(0, 256), slice(0, 7)):               # tiles and the streaming kernel
        y = m.moe_linear(x[rows].contiguous(), eye, activation=name, out_dtype=torch.float32)
        check(name, y, want[rows], (r * U32 * want.abs() + lost_value(v))[rows])


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
def test_slopes(name, dt):
    """Experts of one row each: their bias gradients are the slopes in float32."""
    import extreme_quantized_moe_amd as m
    x = grid(name, dt)
    off = torch.arange(257, dtype=torch.int32, device="cuda")
    _, _, slope = m.moe_linear_act_grad(torch.ones_like(x), x, name, offsets=off, bias_grad=True)
    v = x.to(F64)
    _, r, g = parts(name, v)
    if name == "gelu":
        phi = torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
        bound = g * r + v.abs() * phi * r
    else:
        d = C2 * (1 + 3 * 0.044715 * v * v) if name == "gelu_tanh" else torch.ones_like(v)
        bound = g * r + v.abs() * d * g * ((1 - g) * (r + 4) + 4)
    want = act_slope(name, v)
    check(name, slope, want, U32 * bound + lost_slope(v))
    tail = v < -5
    assert bool((U32 * bound < 1e-4 * want.abs())[tail].all())      # the bound itself is relative there
