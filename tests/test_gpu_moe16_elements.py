"""Every element of the 16-bit layer's output and gradients against float64,
within bounds that follow the layer's own roundings from tensor to tensor.

u is half a step of the 16-bit type.  A stored tensor adds u |value|; a product
carries its operands' errors through the absolute values of the other operand
and adds (depth + 2) roundings of 2^-24 of the sum of absolute products.  SiLU's
slope is at most 1.1, its second derivative at most 0.5.  Second-order terms are
covered by the factor 1.05."""
import pytest
import torch

from tests.moe16_reference import F64, U32, act, act_slope, check, half_step, product_bound, tiny

pytestmark = pytest.mark.gpu

# type, tokens, E, k, S, H, F, renormalized
CASES = [(torch.bfloat16, 5, 8, 2, 0, 64, 96, True), (torch.float16, 33, 6, 3, 2, 136, 72, False),
         (torch.bfloat16, 300, 4, 2, 1, 40, 24, True), (torch.float16, 700, 3, 2, 0, 136, 264, False),
         (torch.bfloat16, 130, 66, 6, 2, 72, 40, False), (torch.float16, 64, 16, 4, 0, 61, 37, True)]


class Val:
    """A float64 tensor and a bound on what the layer's differs from it by."""

    def __init__(self, v, e):
        self.v, self.e = v, e

    def stored(self, dt):
        return Val(self.v, self.e + half_step(dt) * (self.v.abs() + self.e) + tiny(dt))


def times(a, b, depth):
    """a b (matrices)."""
    v = torch.mm(a.v, b.v.contiguous())
    ab, bb = a.v.abs(), b.v.abs().contiguous()
    e = torch.mm(a.e, bb + b.e) + torch.mm(ab, b.e.contiguous())
    return Val(v, e + product_bound(depth, torch.mm(ab, bb)))


def scaled(a, s, es):
    """a times the numbers s (off by es), elementwise with broadcasting."""
    return Val(a.v * s, a.e * s.abs() + (a.v.abs() + a.e) * es + 2 * U32 * (a.v * s).abs())


def plus(a, b):
    return Val(a.v + b.v, a.e + b.e + U32 * (a.v + b.v).abs())


def turned(a):
    return Val(a.v.t().contiguous(), a.e.t().contiguous())


def layer_bounds(dt, x, logits, dout, w1, w3, w2, ids, k, S, renorm):
    """Outputs and gradients as Vals, from the operands alone."""
    def val(t):
        return Val(t.to(F64), torch.zeros(t.shape, dtype=F64, device=t.device))
    T, E = logits.shape
    l = logits.to(F64)
    p = torch.softmax(l.gather(1, ids), 1) if renorm else torch.softmax(l, 1).gather(1, ids)
    ep = (E + 40) * U32 * p
    slots = [(ids[:, j], p[:, j], ep[:, j]) for j in range(k)]
    slots += [(torch.full_like(ids[:, 0], E + s), torch.ones_like(p[:, 0]), torch.zeros_like(p[:, 0])) for s in range(S)]
    dev, H, F = x.device, x.shape[1], w1.shape[1]

    def zero(*shape):
        return Val(torch.zeros(shape, dtype=F64, device=dev), torch.zeros(shape, dtype=F64, device=dev))
    out, dx = zero(T, H), zero(T, H)
    g = zero(T, k + S)
    dw1, dw3, dw2 = zero(E + S, F, H), zero(E + S, F, H), zero(E + S, H, F)
    for e in range(E + S):
        pairs = [(j, t) for j, (who, _, _) in enumerate(slots) for t in torch.nonzero(who == e)[:, 0].tolist()]
        if not pairs:
            continue
        j, t = (torch.tensor(c, device=dev) for c in zip(*pairs))
        w = torch.stack([s[1] for s in slots], 1)[t, j][:, None]
        ew = torch.stack([s[2] for s in slots], 1)[t, j][:, None]
        xs, d = val(x[t]), val(dout[t])
        up = times(xs, turned(val(w3[e])), H).stored(dt)
        pre = times(xs, turned(val(w1[e])), H)
        silu = Val(act("silu", pre.v), 1.1 * pre.e + 128 * U32 * pre.v.abs())
        h = Val(silu.v * up.v, silu.e * (up.v.abs() + up.e) + silu.v.abs() * up.e).stored(dt)
        y = times(h, turned(val(w2[e])), F).stored(dt)
        o = scaled(y, w, ew)
        dots = (d.v * y.v).sum(1)
        g.v[t, j] = dots
        g.e[t, j] = (d.v.abs() * y.e).sum(1) + (H + 2) * U32 * (d.v * y.v).abs().sum(1)
        dy = scaled(d, w, ew).stored(dt)
        dh = times(dy, val(w2[e]), H).stored(dt)
        kept = pre.stored(dt)
        slope = Val(act_slope("silu", pre.v), 0.5 * kept.e + 128 * U32)
        value = Val(silu.v, 1.1 * kept.e + 128 * U32 * pre.v.abs())
        dup = Val(dh.v * value.v, dh.e * (value.v.abs() + value.e) + dh.v.abs() * value.e).stored(dt)
        us = Val(up.v * slope.v, up.e * (slope.v.abs() + slope.e) + up.v.abs() * slope.e)
        dpre = Val(dh.v * us.v, dh.e * (us.v.abs() + us.e) + dh.v.abs() * us.e).stored(dt)
        # the up product's half of dx is rounded to the 16-bit type before the gate's is added
        dxs = plus(times(dpre, val(w1[e]), F), times(dup, val(w3[e]), F).stored(dt)).stored(dt)
        for to, part in ((out, o), (dx, dxs)):
            to.v.index_add_(0, t, part.v)
            to.e.index_add_(0, t, part.e + (k + S) * U32 * part.v.abs())
        n = len(pairs)
        for to, part in ((dw2, times(turned(dy), h, n)), (dw1, times(turned(dpre), xs, n)), (dw3, times(turned(dup), xs, n))):
            to.v[e], to.e[e] = part.v, part.e + U32 * part.v.abs()
    # router: dl_i = p_i (g_i - sum_j p_j g_j)
    gk, ge = g.v[:, :k], g.e[:, :k]
    mean, emean = (p * gk).sum(1, keepdim=True), (p * ge).sum(1, keepdim=True)
    small = (E + 40) * U32 * gk.abs().amax(1, keepdim=True)
    dl, el = torch.zeros_like(l), torch.zeros_like(l)
    if renorm:
        dl.scatter_(1, ids, p * (gk - mean))
        el.scatter_(1, ids, p * (ge + emean + small))
    else:
        q = torch.softmax(l, 1)
        dl = (-q * mean).scatter_add(1, ids, p * gk)
        el = (q * (emean + small)).scatter_add(1, ids, p * (ge + small))
    return dict(out=out.stored(dt), dx=dx.stored(dt), dlogits=Val(dl, el), dw1=dw1, dw3=dw3, dw2=dw2)


def inputs(dt, T, E, k, S, H, F, dev, seed=0):
    gen = torch.Generator().manual_seed(seed + T)
    def rand(*shape, sigma=1.0, t=dt):
        return (torch.randn(shape, generator=gen) * sigma).to(t).to(dev)
    return (rand(T, H), rand(T, E, t=torch.float32), rand(T, H), rand(E + S, F, H, sigma=H ** -0.5),
            rand(E + S, F, H, sigma=H ** -0.5), rand(E + S, H, F, sigma=F ** -0.5))


@pytest.mark.parametrize("dt,T,E,k,S,H,F,renorm", CASES)
def test_every_element(dt, T, E, k, S, H, F, renorm):
    import extreme_quantized_moe_amd as m
    x, logits, dout, w1, w3, w2 = inputs(dt, T, E, k, S, H, F, "cuda")
    lay = m.MoELayer16(w1, w3, w2, E, k, S, renorm)
    out, kept = lay.forward(x, logits, keep=True)
    got = dict(lay.backward(dout, kept, dw_dtype=torch.float32), out=out)
    want = layer_bounds(dt, x, logits, dout, w1, w3, w2, kept["route"]["ids"].long(), k, S, renorm)
    for name, w in want.items():
        # the bound of a whole tensor says something: zeros, or another sign, would not pass
        assert float(w.e.norm()) < 0.6 * float(w.v.norm()), name
        check(name, got[name], w.v, 1.05 * w.e + 1e-30)


@pytest.mark.parametrize("dt,T,E,k,S,H,F,renorm", CASES)
def test_router_gradient_from_what_was_kept(dt, T, E, k, S, H, F, renorm):
    """The way from the experts' rows to the logits' gradient has no 16-bit step: float32 bounds."""
    import extreme_quantized_moe_amd as m
    x, logits, dout, w1, w3, w2 = inputs(dt, T, E, k, S, H, F, "cuda", 7)
    lay = m.MoELayer16(w1, w3, w2, E, k, S, renorm)
    _, kept = lay.forward(x, logits, keep=True)
    got = lay.backward(dout, kept)["dlogits"]
    ids, y = kept["route"]["ids"].long(), kept["y"].to(F64)
    terms = y[kept["route"]["pair_pos"].long()].view(T, k + S, H)[:, :k] * dout.to(F64)[:, None]
    g, eg = terms.sum(2), (H + 2) * U32 * terms.abs().sum(2)
    l = logits.to(F64).requires_grad_(True)
    p = torch.softmax(l.gather(1, ids), 1) if renorm else torch.softmax(l, 1).gather(1, ids)
    (p * g).sum().backward()
    bound = ((E + 40) * U32 * g.abs().amax(1) + 2 * eg.amax(1))[:, None].expand(T, E)
    assert float(bound.norm()) < 0.01 * float(l.grad.norm())
    check("dlogits", got, l.grad, bound)
