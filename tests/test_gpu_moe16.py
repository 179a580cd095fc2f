"""The 16-bit MoE operators as they are used together: routing, dispatch, the
experts' products and the way back, forward and backward, against a float64
layer; captured into a graph and replayed between eager work; on two streams
at once."""
import pytest
import torch

from tests.moe16_reference import F64, act, half_step

pytestmark = pytest.mark.gpu


def _m():
    import extreme_quantized_moe_amd as m
    return m


def rand(shape, dt, seed, sigma=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * sigma).to(dt)


def layer(dt, E, k, S, H, F, renorm=True, seed=0):
    m = _m()
    w1, w3, w2 = (rand((E + S, F, H), dt, seed + 1, H ** -0.5), rand((E + S, F, H), dt, seed + 2, H ** -0.5),
                  rand((E + S, H, F), dt, seed + 3, F ** -0.5))
    return m.MoELayer16(w1, w3, w2, E, k, S, renorm)


def layer_ref(x, logits, w1, w3, w2, ids, S, renorm):
    """The whole layer in float64, differentiable: every expert on every token, weighted."""
    T, E = logits.shape
    p = torch.softmax(logits.gather(1, ids), 1) if renorm else torch.softmax(logits, 1).gather(1, ids)
    gate = torch.zeros((T, E), dtype=F64, device=x.device).scatter(1, ids, p)
    gate = torch.cat([gate, torch.ones((T, S), dtype=F64, device=x.device)], 1)
    out = torch.zeros_like(x)
    for e in range(E + S):
        h = act("silu", torch.mm(x, w1[e].t().contiguous())) * torch.mm(x, w3[e].t().contiguous())
        out = out + gate[:, e:e + 1] * torch.mm(h, w2[e].t().contiguous())
    return out


CASES = [(torch.bfloat16, 5, 8, 2, 0, 64, 96, True), (torch.float16, 33, 6, 3, 2, 136, 72, False),
         (torch.bfloat16, 300, 4, 2, 1, 264, 328, True), (torch.float16, 1, 3, 1, 0, 61, 37, True),
         (torch.float16, 700, 2, 2, 0, 256, 512, False)]


def rel(a, b):
    return float((a.to(F64) - b).norm() / b.norm().clamp(min=1e-300))


@pytest.mark.parametrize("dt,T,E,k,S,H,F,renorm", CASES)
def test_layer_forward_and_gradients(dt, T, E, k, S, H, F, renorm):
    lay = layer(dt, E, k, S, H, F, renorm)
    x, logits, dout = rand((T, H), dt, 11), rand((T, E), torch.float32, 12), rand((T, H), dt, 13)
    out, kept = lay.forward(x, logits, keep=True)
    assert torch.equal(out, lay.forward(x, logits))
    grads = lay.backward(dout, kept, dw_dtype=torch.float32)
    leaves = [t.to(F64).requires_grad_(True) for t in (x, logits, lay.w1, lay.w3, lay.w2)]
    ref = layer_ref(*leaves, kept["route"]["ids"].long(), S, renorm)
    want = torch.autograd.grad((ref * dout.to(F64)).sum(), leaves)
    # Each stored intermediate is off by at most half a step u of its type,
    # independently; in Frobenius norm the way to a result adds at most one u
    # (times a factor under 2 for the activation and the gate product) per
    # stored tensor: up, h, y, out forward; dy, dh, dpre, dup, dx parts on the
    # way back with the forward ones read again.
    u = half_step(dt)
    assert rel(out, ref.detach()) <= 2 * 4 * u
    for name, g, w in zip(("dx", "dlogits", "dw1", "dw3", "dw2"), (grads[n] for n in ("dx", "dlogits", "dw1", "dw3", "dw2")),
                          want):
        if float(w.norm()) < 1e-12:       # one pick renormalized: its weight is constant
            assert float(g.double().norm()) < 1e-4 * T, name
            continue
        # dlogits is a difference of dot products: its part that cancels is bounded through the dots' norm
        scale = 1.0
        if name == "dlogits":
            full = torch.autograd.grad((layer_ref(*leaves, kept["route"]["ids"].long(), S, renorm) * dout.to(F64)).sum(),
                                       leaves[1])[0]
            scale = max(1.0, float(ref.detach().norm() * dout.double().norm() / T ** 0.5 / full.norm()))
        assert rel(g, w) <= 2 * 9 * u * scale, name


def test_layer_gradients_against_differences():
    """Directional derivatives of the float64 layer by central differences."""
    dt = torch.float16
    lay = layer(dt, 4, 2, 1, 72, 88)
    x, logits, dout = rand((20, 72), dt, 1), rand((20, 4), torch.float32, 2), rand((20, 72), dt, 3)
    out, kept = lay.forward(x, logits, keep=True)
    g = lay.backward(dout, kept, dw_dtype=torch.float32)
    base = [t.to(F64) for t in (x, logits, lay.w1, lay.w3, lay.w2)]
    ids = kept["route"]["ids"].long()

    def f(args):
        return float((layer_ref(*args, ids, 1, True) * dout.to(F64)).sum())
    for i, name in enumerate(("dx", "dlogits", "dw1", "dw3", "dw2")):
        u = g[name].to(F64)                       # along the gradient itself: the derivative is its squared norm
        h = 1e-6 / float(u.abs().max())
        moved = [list(base), list(base)]
        moved[0][i], moved[1][i] = base[i] + h * u, base[i] - h * u
        diff = (f(moved[0]) - f(moved[1])) / (2 * h)
        assert abs(diff - float((u * u).sum())) <= 2 * 9 * half_step(dt) * float((u * u).sum()) * 2, name


def test_router_product_feeds_the_layer():
    """Logits from the router's own 16-bit product in 32 bits, and its gradients."""
    m = _m()
    dt = torch.bfloat16
    lay = layer(dt, 8, 2, 0, 128, 64)
    x, wg = rand((50, 128), dt, 1), rand((8, 128), dt, 2, 0.1)
    logits = m.moe_linear(x, wg, out_dtype=torch.float32)
    out, kept = lay.forward(x, logits, keep=True)
    g = lay.backward(rand((50, 128), dt, 3), kept)
    dx, dwg = m.moe_linear_grad(g["dlogits"].to(dt), x, wg, dx_add=g["dx"])
    want = torch.mm(g["dlogits"].to(dt).to(F64).t().contiguous(), x.to(F64))
    assert rel(dwg, want) <= half_step(dt) * 1.01
    assert rel(dx, torch.mm(g["dlogits"].to(dt).to(F64), wg.to(F64)) + g["dx"].to(F64)) <= half_step(dt) * 1.01


def test_captured_and_replayed():
    """Forward and backward in one graph, replayed with new inputs between
    eager calls of the same layer; a second graph of the same calls beside it."""
    dt = torch.bfloat16
    lay = layer(dt, 8, 2, 1, 264, 136)
    T = 37
    x, logits, dout = rand((T, 264), dt, 1), rand((T, 8), torch.float32, 2), rand((T, 264), dt, 3)

    def step():
        out, kept = lay.forward(x, logits, keep=True)
        g = lay.backward(dout, kept, dw_dtype=torch.float32)
        return [out] + [g[n] for n in ("dx", "dlogits", "dw1", "dw3", "dw2")]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step())
        graphs.append(g)
    for i in range(4):
        x.copy_(rand((T, 264), dt, 20 + i))
        logits.copy_(rand((T, 8), torch.float32, 30 + i))
        dout.copy_(rand((T, 264), dt, 40 + i))
        want = step()
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        for a, b in zip(outs[i % 2], want):
            assert torch.equal(a, b)
        graphs[1 - i % 2].replay()
        again = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs[1 - i % 2], again))


def test_two_streams_at_once():
    """Calls on two streams share nothing: the results are the one-stream results."""
    m = _m()
    dt = torch.bfloat16
    x, w, dy = rand((200, 2048), dt, 1), rand((64, 2048), dt, 2, 0.02), rand((200, 64), dt, 3)
    pre = rand((200, 64), dt, 4)

    def work(a):
        return [m.moe_linear(a, w, activation="gelu"), *m.moe_linear_grad(dy, a, w),
                m.moe_linear_act_grad(dy, pre, "gelu", bias_grad=True)[2]]
    xs = [x, (x.float() * 0.5).to(dt)]
    want = [work(a) for a in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(work(xs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))


def test_layer_refuses_other_logits():
    lay = layer(torch.bfloat16, 4, 2, 0, 64, 32)
    x = rand((6, 64), torch.bfloat16, 1)
    for bad in (rand((6, 4), torch.bfloat16, 2), rand((6, 5), torch.float32, 2), rand((5, 4), torch.float32, 2)):
        with pytest.raises(ValueError):
            lay.forward(x, bad)
    with pytest.raises(ValueError):
        lay.forward(x.half(), rand((6, 4), torch.float32, 2))


def test_layer_on_two_streams_at_once():
    """Two layers' passes overlap on two streams: routing scratch and all else are each call's own."""
    dt = torch.bfloat16
    lays = [layer(dt, 8, 2, 0, 256, 128, seed=s) for s in (0, 10)]
    ins = [(rand((2000, 256), dt, 5 + s), rand((2000, 8), torch.float32, 7 + s), rand((2000, 256), dt, 9 + s))
           for s in (0, 10)]

    def work(i):
        out, kept = lays[i].forward(*ins[i][:2], keep=True)
        g = lays[i].backward(ins[i][2], kept)
        return [out, *(g[n] for n in ("dx", "dlogits", "dw1", "dw3", "dw2"))]
    want = [work(0), work(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(work(i))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))
