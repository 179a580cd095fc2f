"""Grouped products with more than 2^31 weights, weight gradients or results:
the last experts, rows and columns against float64."""
import pytest
import torch

from tests.moe16_reference import F64, U32, check, linear_ref, product_bound, rounded

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _m():
    import extreme_quantized_moe_amd as m
    return m


def rand(shape, sigma=1.0, seed=1):
    """bf16 values, a part at a time (the largest tensors have 4e9)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = torch.empty(shape, dtype=BF16, device="cuda")
    flat = out.view(-1)
    for a in range(0, flat.numel(), 1 << 28):
        part = flat[a:a + (1 << 28)]
        part.copy_(torch.randn(part.shape, generator=g, device="cuda") * sigma)
    return out


@pytest.mark.parametrize("N,K", [(4096, 3584), (3583, 4097)])
@pytest.mark.parametrize("rows", [1, 37])
def test_weights_over_31_bits(N, K, rows):
    """256 experts: 3.7e9 weights, `rows` rows for each of a fifth of them."""
    m = _m()
    E = 256
    counts = [rows if e % 5 == 0 or e >= 250 else 0 for e in range(E)]
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1:] = torch.tensor(counts, device="cuda").cumsum(0)
    bounds = off.tolist()
    R = bounds[-1]
    w = rand((E, N, K), K ** -0.5)
    x, dy = rand((R, K), seed=2), rand((R, N), seed=3)
    y = m.moe_linear(x, w, off, activation="relu", max_rows_per_expert=rows)
    dx, dw = m.moe_linear_grad(dy, x, w, off)
    for e in (0, 150, 250, 255):
        a, b = bounds[e], bounds[e + 1]
        xe, de, we = x[a:b], dy[a:b].to(F64), w[e].to(F64)
        want, _, err, _ = linear_ref(xe, w[e:e + 1], [0, b - a], None, "relu", None, None)
        check(f"y of expert {e}", y[a:b], want, err + rounded(want, BF16))
        want = torch.mm(de, we)
        check(f"dx of expert {e}", dx[a:b], want, product_bound(N, torch.mm(de.abs(), we.abs())) + rounded(want, BF16))
        dt, xd = de.t().contiguous(), xe.to(F64)
        want = torch.mm(dt, xd)
        check(f"dw of expert {e}", dw[e], want, product_bound(b - a, torch.mm(dt.abs(), xd.abs())) + rounded(want, BF16))
    assert not dw[1].any() and not dw[249].any()       # experts without a row


@pytest.mark.parametrize("N", [2304, 2303])
def test_results_over_31_bits(N):
    """2^20 rows of 2304 results, with everything of that size in the epilogue."""
    m = _m()
    R, K = 1 << 20, 64
    x, w = rand((R, K)), rand((1, N, K), K ** -0.5, 2)
    mul, res = rand((R, N), seed=3), rand((R, N), seed=4)
    y, pre = m.moe_linear(x, w, activation="silu", mul=mul, residual=res, return_pre=True)
    dpre, dmul, db = m.moe_linear_act_grad(y, pre, "silu", mul=mul, bias_grad=True)
    plain, _, _ = m.moe_linear_act_grad(y, pre, "silu", mul=mul)
    assert torch.equal(plain[-4096:], dpre[-4096:])
    del plain
    dx, _ = m.moe_linear_grad(dpre, x, w, need_dw=False)
    for a in (0, R // 2 - 100, R - 200):
        s = slice(a, a + 200)
        want, wpre, err, perr = linear_ref(x[s], w, [0, 200], None, "silu", mul[s], res[s])
        check("y", y[s], want, err + rounded(want, BF16))
        check("pre", pre[s], wpre, perr + rounded(wpre, BF16))
        p, d = pre[s].to(F64), y[s].to(F64)
        g = torch.sigmoid(p)
        want = d * p * g
        check("dmul", dmul[s], want, 130 * U32 * want.abs() + rounded(want, BF16))
        want = d * mul[s].to(F64) * (g + p * g * (1 - g))
        check("dpre", dpre[s], want, 128 * U32 * 1.2 * (d * mul[s].to(F64)).abs() + rounded(want, BF16))
        dd, wd = dpre[s].to(F64), w[0].to(F64)
        want = torch.mm(dd, wd)
        check("dx", dx[s], want, product_bound(N, torch.mm(dd.abs(), wd.abs())) + rounded(want, BF16))
    # weight gradients of the last rows alone: the others are zeros
    x[:-4096] = 0
    _, dw = m.moe_linear_grad(dpre, x, w, need_dx=False, dw_dtype=torch.float32)
    dd, xd = dpre[-4096:].to(F64).t().contiguous(), x[-4096:].to(F64)
    check("dw", dw[0], torch.mm(dd, xd), product_bound(4096, torch.mm(dd.abs(), xd.abs())) + 1e-30)
