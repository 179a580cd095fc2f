"""The grouped 16-bit product with its epilogue and its gradients on the GPU
against float64: experts without rows, one row, ragged and odd sizes, operands
off a 16-byte address, every epilogue, rows outside the table left as they
were, values that must not leak between experts."""
import pytest
import torch

from tests.moe16_reference import (F64, U32, act, act_slope, check, linear_ref, lost_slope, lost_value,
                                   product_bound, rounded, spans)

pytestmark = pytest.mark.gpu
TYPES = [torch.float16, torch.bfloat16]


def _m():
    import extreme_quantized_moe_amd as m
    return m


def rand(shape, dt, seed, sigma=1.0, offset=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = 1
    for s in shape:
        n *= s
    return (torch.randn(n + offset, generator=g, device="cuda") * sigma).to(dt)[offset:].view(shape)


def table(counts, lead=0):
    off = [lead]
    for c in counts:
        off.append(off[-1] + c)
    return off, torch.tensor(off, dtype=torch.int32, device="cuda")


# rows of each expert, N, K
SHAPES = [
    ([1], 1, 1), ([1], 16, 8), ([1], 64, 64), ([1], 4096, 512), ([1], 130, 4104), ([3], 65, 33), ([16], 128, 128),
    ([17], 264, 72), ([33], 1, 520), ([64], 64, 2048), ([65], 63, 65), ([130], 200, 96), ([257], 8, 1000),
    ([300], 520, 136), ([0], 32, 32), ([0, 0, 5], 48, 40), ([1, 0, 2, 1], 256, 512), ([4, 3, 0, 9], 1416, 264),
    ([17, 1, 40, 0, 64], 136, 200), ([70, 0, 129, 3], 264, 328), ([31, 33], 129, 127), ([256, 256], 256, 256),
    ([300, 1, 520], 384, 192), ([5] * 66, 72, 64), ([2, 0, 1] * 40, 24, 16), ([1000, 24], 512, 1032),
    ([15, 16, 17, 31, 32, 33], 2056, 1096), ([700], 1024, 2048), ([90, 40], 5000, 64),
    ([300, 0, 200], 515, 1031), ([700], 331, 2049), ([4, 1, 9], 1001, 4099), ([1], 4097, 130), ([200], 50, 1999),
    ([100], 384, 4096), ([129, 385], 264, 1544),
]
EPILOGUES = [  # bias, activation, mul, residual, out fp32, keep
    (False, "none", False, False, False, False), (True, "relu", False, True, False, True),
    (False, "silu", True, False, False, True), (True, "gelu", False, False, True, False),
    (True, "gelu_tanh", True, True, False, False), (False, "none", False, True, True, False),
]


def linear_case(dt, counts, N, K, epi, offset=0, lead=0, tail=0, use_table=True):
    bias, name, mul, res, f32, keep = epi
    off, dev = table(counts, lead)
    R, E = off[-1] + tail, len(counts)
    x, w = rand((R, K), dt, 1, 1.0, offset), rand((E, N, K), dt, 2, K ** -0.5, offset)
    b = rand((E, N), dt, 3, 0.5, offset) if bias else None
    mu = rand((R, N), dt, 4, 1.0, offset) if mul else None
    re = rand((R, N), dt, 5, 1.0, offset) if res else None
    x[:lead] = float("nan")
    x[off[-1]:] = float("inf")
    odt = torch.float32 if f32 else dt
    out = torch.full((R * N + offset,), 7.0, dtype=odt, device="cuda")[offset:].view(R, N)
    got = _m().moe_linear(x, w, dev if use_table else None, bias=b, activation=name, mul=mu, residual=re,
                          out_dtype=odt, return_pre=keep, out=out)
    y, pre = got if keep else (got, None)
    inside = slice(lead, off[-1])
    xr = torch.where(torch.isfinite(x.float()), x, torch.zeros_like(x))
    want, wpre, err, perr = linear_ref(xr, w, off, b, name, mu, re)
    check("y", y[inside], want[inside], err[inside] + (rounded(want, dt)[inside] if not f32 else U32 * want[inside].abs())
          + 1e-30)
    if keep:
        check("pre", pre[inside], wpre[inside], perr[inside] + rounded(wpre, dt)[inside])
    for outside in (y[:lead], y[off[-1]:]):
        assert torch.equal(outside, torch.full_like(outside, 7.0)), "rows outside the table were written"


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("counts,N,K", SHAPES)
def test_sizes(dt, counts, N, K):
    i = (N + K + len(counts)) % len(EPILOGUES)
    linear_case(dt, counts, N, K, EPILOGUES[i])
    linear_case(dt, counts, N, K, EPILOGUES[(i + 1) % len(EPILOGUES)])


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("epi", EPILOGUES)
@pytest.mark.parametrize("counts,N,K", [([5], 264, 520), ([70, 0, 200], 264, 136), ([9, 1, 0, 30], 63, 37),
                                        ([600], 64, 1024)])
def test_epilogues(dt, epi, counts, N, K):
    linear_case(dt, counts, N, K, epi)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("offset", [1, 2, 4])
@pytest.mark.parametrize("counts", [[3, 5], [100, 90]])
def test_operands_off_a_16_byte_address(dt, offset, counts):
    linear_case(dt, counts, 128, 192, EPILOGUES[4], offset=offset)


@pytest.mark.parametrize("counts", [[2, 0, 3], [64, 1, 130], [300, 300]])
@pytest.mark.parametrize("N,K", [(128, 256), (130, 31)])
def test_rows_outside_the_table(counts, N, K):
    for epi in (EPILOGUES[2], EPILOGUES[1]):
        linear_case(torch.bfloat16, counts, N, K, epi, lead=3, tail=5)


def test_one_expert_without_a_table():
    for R in (1, 40, 500):
        linear_case(torch.float16, [R], 256, 320, EPILOGUES[4], use_table=False)


def test_large_row_counts_of_one_expert():
    """More than one wave of tiles over the chip, all compared."""
    linear_case(torch.bfloat16, [2900, 0, 1300], 2056, 520, EPILOGUES[2])
    linear_case(torch.float16, [4500], 4104, 264, EPILOGUES[1])


def test_row_bound_only_steers():
    """A row bound that is too small costs speed, never rows."""
    m = _m()
    x, w = rand((300, 256), torch.bfloat16, 1), rand((2, 264, 256), torch.bfloat16, 2, 0.06)
    off = torch.tensor([0, 40, 300], dtype=torch.int32, device="cuda")
    want, _, err, _ = linear_ref(x, w, [0, 40, 300], None, "none", None, None)
    for bound in (0, 1, 16, 64, 300, 100000):
        y = m.moe_linear(x, w, off, max_rows_per_expert=bound)
        check(f"bound {bound}", y, want, err + rounded(want, torch.bfloat16))


def test_values_stay_with_their_expert():
    """Non-finite rows, weights and gradients of one expert reach no other."""
    m = _m()
    for dt, N, K in ((torch.bfloat16, 264, 328), (torch.float16, 77, 61)):
        off, dev = table([40, 70, 5])
        x, w, dy = rand((115, K), dt, 1), rand((3, N, K), dt, 2, 0.05), rand((115, N), dt, 3)
        clean_y, (clean_dx, clean_dw) = m.moe_linear(x, w, dev), m.moe_linear_grad(dy, x, w, dev)
        x[40:110], dy[40:110], w[1] = float("nan"), float("inf"), float("nan")
        y, (dx, dw) = m.moe_linear(x, w, dev), m.moe_linear_grad(dy, x, w, dev)
        for a, b in ((y, clean_y), (dx, clean_dx)):
            assert torch.equal(a[:40], b[:40]) and torch.equal(a[110:], b[110:])
            assert torch.isnan(a[40:110].float()).all()
        assert torch.equal(dw[0], clean_dw[0]) and torch.equal(dw[2], clean_dw[2])


def test_offsets_are_clipped():
    """A table past the buffer reads and writes nothing outside it."""
    m = _m()
    x, w = rand((50, 64), torch.float16, 1), rand((3, 72, 64), torch.float16, 2, 0.1)
    off = torch.tensor([-5, 20, 20, 1 << 30], dtype=torch.int32, device="cuda")
    y = m.moe_linear(x, w, off)
    want, _, err, _ = linear_ref(x, w, [0, 20, 20, 50], None, "none", None, None)
    check("y", y, want, err + rounded(want, torch.float16))
    dx, dw = m.moe_linear_grad(y, x, w, off)
    dx2, dw2 = m.moe_linear_grad(y, x, w, torch.tensor([0, 20, 20, 50], dtype=torch.int32, device="cuda"))
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


def test_residual_and_gate_buffers_may_be_the_output():
    m = _m()
    for R, N in ((9, 264), (300, 264), (40, 61)):
        x, w = rand((R, 128), torch.bfloat16, 1), rand((N, 128), torch.bfloat16, 2, 0.1)
        res = rand((R, N), torch.bfloat16, 3)
        a = m.moe_linear(x, w, residual=res)
        b = m.moe_linear(x, w, mul=res)
        own = res.clone()
        assert torch.equal(m.moe_linear(x, w, residual=own, out=own), a)
        own = res.clone()
        assert torch.equal(m.moe_linear(x, w, mul=own, out=own), b)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("counts,N,K", SHAPES)
def test_product_gradients(dt, f32, counts, N, K):
    m = _m()
    off, dev = table(counts, lead=2)
    R, E = off[-1] + 3, len(counts)
    x, w, dy = rand((R, K), dt, 1), rand((E, N, K), dt, 2, 0.1), rand((R, N), dt, 3)
    x[:2], x[off[-1]:], dy[:2], dy[off[-1]:] = (float("nan"),) * 4
    add = rand((R, K), dt, 4) if (N + K) % 2 else None
    dx, dw = m.moe_linear_grad(dy, x, w, dev, dw_dtype=torch.float32 if f32 else dt, dx_add=add)
    wdx, mag = torch.zeros((R, K), dtype=F64, device="cuda"), torch.zeros((R, K), dtype=F64, device="cuda")
    wdw, mdw = torch.zeros((E, N, K), dtype=F64, device="cuda"), torch.zeros((E, N, K), dtype=F64, device="cuda")
    for e, (a, b) in enumerate(spans(off)):
        d, we, xe = dy[a:b].to(F64), w[e].to(F64), x[a:b].to(F64)
        wdx[a:b], mag[a:b] = torch.mm(d, we), torch.mm(d.abs(), we.abs())
        dt_ = d.t().contiguous()
        wdw[e], mdw[e] = torch.mm(dt_, xe), torch.mm(dt_.abs(), xe.abs())
    s = slice(2, off[-1])
    if add is not None:
        wdx[s] += add[s].to(F64)
        mag[s] += add[s].to(F64).abs()
    check("dx", dx[s], wdx[s], product_bound(N + 1, mag[s]) + rounded(wdx[s], dt))
    most = max(counts)
    check("dw", dw, wdw, product_bound(most, mdw) + (U32 * wdw.abs() + 1e-30 if f32 else rounded(wdw, dt)))
    only_dx = m.moe_linear_grad(dy, x, w, dev, need_dw=False, dx_add=add)
    only_dw = m.moe_linear_grad(dy, x, w, dev, need_dx=False, dw_dtype=torch.float32 if f32 else dt)
    assert only_dx[1] is None and torch.equal(only_dx[0][s], dx[s])
    assert only_dw[0] is None and torch.equal(only_dw[1], dw)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("name", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("counts,N,offset", [([5], 8, 0), ([40, 0, 70], 264, 0), ([1, 33, 2], 61, 0), ([65, 64], 1030, 0),
                                             ([300], 72, 1), ([0, 0], 16, 0), ([1100, 3], 40, 0)])
def test_activation_gradients(dt, name, gated, counts, N, offset):
    m = _m()
    off, dev = table(counts, lead=1)
    R, E = off[-1] + 2, len(counts)
    dy, pre = rand((R, N), dt, 1, 1.0, offset), rand((R, N), dt, 2, 3.0, offset)
    mul = rand((R, N), dt, 3, 1.0, offset) if gated else None
    outside = [0, R - 2, R - 1]
    dy[outside] = float("nan")
    s = slice(1, off[-1])
    v, d = pre.to(F64), dy.to(F64)
    mu = mul.to(F64) if gated else torch.ones_like(v)
    slope, value = act_slope(name, v), act(name, v)
    # float32: tens of roundings of the activation (bounded like the forward
    # value); the slope's two terms are each at most 1.5 and may cancel
    wpre = d * mu * slope
    err = 128 * U32 * (d * mu).abs() * (slope.abs() + (v * value).abs().clamp(max=1) + 1e-3) \
        + lost_slope(v) * (d * mu).abs() if name not in ("none", "relu") else 4 * U32 * wpre.abs()
    for bias in (False, True):
        dpre, dmul, dbias = m.moe_linear_act_grad(dy, pre, name, mul=mul, offsets=dev, bias_grad=bias)
        check("dpre", dpre[s], wpre[s], err[s] + rounded(wpre[s], dt))
        if gated:
            wm = d * value
            check("dmul", dmul[s], wm[s], 130 * U32 * wm[s].abs() + rounded(wm[s], dt) + (lost_value(v) * d.abs())[s])
        else:
            assert dmul is None
        if bias:
            want = torch.stack([wpre[a:b].sum(0) for a, b in spans(off)])
            mag = torch.stack([wpre[a:b].abs().sum(0) for a, b in spans(off)])
            errs = torch.stack([err[a:b].sum(0) for a, b in spans(off)])
            check("dbias", dbias, want, errs + (max(counts) + 2) * U32 * mag + 1e-30)
        else:
            assert dbias is None


def test_activation_tails():
    """Far negative and positive arguments, infinities and the lowest values
    keep their limits; the value is right to the type's precision."""
    m = _m()
    eye = torch.eye(16, dtype=torch.bfloat16, device="cuda")
    pts = [0.0, -0.0, 1e-4, -1e-4, -3.0, -4.5, -5.0, -6.0, -9.0, 9.0, 88.0, -88.0, 200.0, -200.0, 3e38, -3e38]
    x = torch.tensor([pts], dtype=torch.bfloat16, device="cuda")
    v = x.to(F64)
    for name in ("relu", "silu", "gelu", "gelu_tanh"):
        y = m.moe_linear(x, eye, activation=name, out_dtype=torch.float32)
        want = torch.nan_to_num(act(name, v.clamp(min=-1e3)))
        check(name, torch.where(v > 1e30, torch.zeros_like(y), y), torch.where(v > 1e30, torch.zeros_like(want), want),
              160 * U32 * want.abs() + lost_value(v.clamp(-1e3, 1e3)) + 1e-45)
        assert float(y[0, 14]) > 2.9e38
        g = torch.ones_like(x)
        dpre, _, _ = m.moe_linear_act_grad(g, x, name)
        slope = act_slope(name, v.clamp(-1e3, 1e3))
        check(name + " slope", dpre, slope, rounded(slope, torch.bfloat16) + 128 * U32 + lost_slope(v.clamp(-1e3, 1e3)))
        inf = torch.tensor([[float("inf"), float("-inf"), float("nan")]], dtype=torch.bfloat16, device="cuda")
        d, _, _ = m.moe_linear_act_grad(torch.ones_like(inf), inf, name)
        assert float(d[0, 0]) == 1.0 and float(d[0, 1]) == 0.0 and torch.isnan(d[0, 2])


def test_results_repeat_bit_for_bit():
    m = _m()
    off, dev = table([300, 0, 41, 700])
    x, w, dy = rand((1041, 1032), torch.bfloat16, 1), rand((4, 520, 1032), torch.bfloat16, 2, 0.05), rand(
        (1041, 520), torch.bfloat16, 3)
    first = (m.moe_linear(x, w, dev), *m.moe_linear_grad(dy, x, w, dev),
             m.moe_linear_act_grad(dy, dy, "gelu", offsets=dev, bias_grad=True)[2])
    for _ in range(3):
        again = (m.moe_linear(x, w, dev), *m.moe_linear_grad(dy, x, w, dev),
                 m.moe_linear_act_grad(dy, dy, "gelu", offsets=dev, bias_grad=True)[2])
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_binding_refusals():
    m = _m()
    x, w = rand((8, 64), torch.bfloat16, 1), rand((2, 32, 64), torch.bfloat16, 2)
    off = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    bad = [dict(offsets=None), dict(offsets=off[:2]), dict(offsets=off.long()), dict(activation="tanh"),
           dict(bias=rand((32,), torch.bfloat16, 3)), dict(bias=rand((2, 32), torch.float16, 3)),
           dict(mul=rand((8, 31), torch.bfloat16, 3)), dict(residual=rand((7, 32), torch.bfloat16, 3)),
           dict(out_dtype=torch.float16), dict(out=torch.empty((8, 33), dtype=torch.bfloat16, device="cuda")),
           dict(offsets=off.cpu())]
    for change in bad:
        with pytest.raises(ValueError):
            m.moe_linear(x, w, **{"offsets": off, **change})
    for args in ((x, w.half(), off), (x[:, :63], w, off), (x.t(), w, off), (x.float(), w, off),
                 (x, w[:, :, :32], off), (x, w.cpu(), off)):
        with pytest.raises(ValueError):
            m.moe_linear(*args)
    with pytest.raises(ValueError):
        m.moe_linear_grad(rand((8, 31), torch.bfloat16, 1), x, w, off)
    with pytest.raises(ValueError):
        m.moe_linear_act_grad(x, x[:4], "silu")
    with pytest.raises(ValueError):
        m.moe_permute(x, off, 3)


@pytest.mark.parametrize("E", [1, 5])
@pytest.mark.parametrize("N,K", [(64, 128), (33, 17)])
def test_no_rows_at_all(E, N, K):
    """A buffer without a row: outputs without a row, weight and bias gradients of zeros."""
    m = _m()
    dt = torch.bfloat16
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    x, w, dy = rand((0, K), dt, 1), rand((E, N, K), dt, 2), rand((0, N), dt, 3)
    assert m.moe_linear(x, w, off, activation="silu").shape == (0, N)
    dx, dw = m.moe_linear_grad(dy, x, w, off, dw_dtype=torch.float32)
    assert dx.shape == (0, K) and torch.equal(dw, torch.zeros_like(dw))
    dpre, _, dbias = m.moe_linear_act_grad(dy, dy, "gelu", offsets=off, bias_grad=True)
    assert dpre.shape == (0, N) and torch.equal(dbias, torch.zeros((E, N), device="cuda"))


@pytest.mark.parametrize("counts,N,K", [([9, 0, 3], 512, 1024), ([700], 64, 1024), ([100], 384, 4096), ([900, 40, 0, 800], 2048, 512),
                                        ([2100, 2000], 2048, 192), ([150, 3], 131, 1031), ([200], 50, 1999)])
def test_every_form_captured(counts, N, K):
    """Streaming, router, split, tile and loose forms in a graph, replayed with
    other inputs between eager calls."""
    m = _m()
    dt = torch.bfloat16
    off, dev = table(counts)
    R, E = off[-1], len(counts)
    x, w, dy = rand((R, K), dt, 1), rand((E, N, K), dt, 2, K ** -0.5), rand((R, N), dt, 3)

    def step():
        y, pre = m.moe_linear(x, w, dev, activation="gelu", residual=dy, return_pre=True)
        dpre, _, db = m.moe_linear_act_grad(dy, pre, "gelu", offsets=dev, bias_grad=True)
        return [y, pre, dpre, db, *m.moe_linear_grad(dpre, x, w, dev, dw_dtype=torch.float32)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for i in range(3):
        x.copy_(rand((R, K), dt, 50 + i))
        dy.copy_(rand((R, N), dt, 60 + i))
        g.replay()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
