"""Float64 definitions of the 16-bit MoE operators and the error bounds their
tests use.

Bounds, per element: u = half a rounding step of the output type relative to
the value (bf16 2^-8 / 2 ... stated as `torch.finfo(t).eps / 2`), plus the
smallest subnormal step for fp16 (values under its normal range), plus float32
work: a sum of n products rounds at most n times, each by 2^-24 of the partial
sum, which the sum of absolute products bounds.

Far tails: the activations are v g and slopes g (1 + ...) with g = c exp(-s),
c <= 1, in float32.  The hardware's exponential returns 0 for results under
2^-126, so g may lose up to 2^-126 there and nowhere else, and what multiplies g
bounds the loss: |v| for the value, (1 + |v|) 2 (1 + v^2) for the slope (the
widest, GELU_TANH: 1 + v (1 - g) 2 sqrt(2/pi) (1 + 0.134 v^2))."""
import math

import torch

U32 = 2.0 ** -24
F64 = torch.float64


def half_step(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    """Half the spacing of the subnormal values of t."""
    return 2.0 ** -25 if t == torch.float16 else torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2


def rounded(value, t):
    """How far one rounding to t can be from `value`."""
    return value.abs() * half_step(t) + tiny(t)


FLUSH = 2.0 ** -126


def lost_value(v):
    return FLUSH * v.abs()


def lost_slope(v):
    return FLUSH * (1 + v.abs()) * 2 * (1 + v * v)


def act(name, v):
    if name == "relu":
        return torch.clamp(v, min=0)
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu":
        return 0.5 * v * torch.erfc(-v / math.sqrt(2))
    if name == "gelu_tanh":
        return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    return v


def act_slope(name, v):
    if name == "relu":
        return (v > 0).to(F64)
    if name == "silu":
        g = torch.sigmoid(v)
        return g + v * g * torch.sigmoid(-v)
    if name == "gelu":
        return 0.5 * torch.erfc(-v / math.sqrt(2)) + v * torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        g = torch.sigmoid(2 * c * (v + 0.044715 * v ** 3))
        return g + v * g * (1 - g) * 2 * c * (1 + 3 * 0.044715 * v * v)
    return torch.ones_like(v)


def check(what, got, want, bound):
    got = got.to(F64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    off = (got - want).abs()
    bad = off > bound
    if bad.any():
        i = int(torch.argmax((off / bound).flatten()))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound, worst at {i}: "
                             f"{float(got.flatten()[i])} want {float(want.flatten()[i])} "
                             f"bound {float(bound.flatten()[i])}")


def spans(offsets):
    return list(zip(offsets, offsets[1:]))


def product_bound(depth, magnitude):
    """Float32 error of sums of `depth` products whose absolute values add up to `magnitude`."""
    return (depth + 2) * U32 * magnitude


def linear_ref(x, w, offsets, bias, name, mul, res):
    """(y, pre, float32 error bound of y, of pre) in float64 for rows inside the offsets."""
    R, N = x.shape[0], w.shape[1]
    pre = torch.zeros((R, N), dtype=F64, device=x.device)
    mag = torch.zeros_like(pre)
    for e, (a, b) in enumerate(spans(offsets)):
        xe, we = x[a:b].to(F64), w[e].to(F64).t().contiguous()
        pre[a:b] = torch.mm(xe, we)
        mag[a:b] = torch.mm(xe.abs(), we.abs())
        if bias is not None:
            pre[a:b] += bias[e].to(F64)
            mag[a:b] += bias[e].to(F64).abs()
    pre_err = product_bound(x.shape[1] + 1, mag)
    y = act(name, pre)
    # slopes stay under 1.13; the float32 activation itself is good to a few
    # tens of roundings (exp of a rounded argument up to ~100: 2^-24 * 100)
    err = 1.13 * pre_err + (0 if name in ("none", "relu") else 128 * U32 * y.abs() + lost_value(pre))
    if mul is not None:
        y = y * mul.to(F64)
        err = err * mul.to(F64).abs() + U32 * y.abs()
    if res is not None:
        y = y + res.to(F64)
        err = err + U32 * (y.abs() + res.to(F64).abs())
    return y, pre, err, pre_err
