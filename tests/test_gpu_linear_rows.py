"""The grouped 16-bit product where rows start off a 16-byte address and there
are rows enough that the operands are copied into whole rows first, or only the
results' rows are odd: against float64, on every epilogue, off an aligned
address, with the contraction split, captured, and with values next to a row's
end that must not reach its results."""
import pytest
import torch

from tests import test_gpu_linear as base
from tests.moe16_reference import F64, check, product_bound, rounded, spans

pytestmark = pytest.mark.gpu
TYPES = base.TYPES

# rows of each expert, N, K: odd N, odd K, both, row lengths of 2 and 4 mod 8
SHAPES = [
    ([2048], 2047, 1024), ([2048], 1024, 1025), ([1500, 0, 700], 1031, 2049), ([260], 4097, 520), ([900], 517, 4098),
    ([3000, 1, 257], 772, 515), ([4000], 257, 129), ([640], 2050, 2046), ([300, 0, 1, 500], 2564, 1284),
    ([1025], 1793, 64), ([8192], 100, 331), ([0, 2600], 263, 777), ([16, 8, 5], 2047, 4098), ([12], 1021, 8191),
    ([1200] * 3, 1409, 513), ([512], 513, 6145), ([8200], 4097, 4099), ([2100] * 4, 2049, 4100),
]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("counts,N,K", SHAPES)
def test_forward(dt, counts, N, K):
    i = (N + K) % len(base.EPILOGUES)
    base.linear_case(dt, counts, N, K, base.EPILOGUES[i])
    base.linear_case(dt, counts, N, K, base.EPILOGUES[(i + 3) % len(base.EPILOGUES)], lead=2, tail=3)


@pytest.mark.parametrize("epi", base.EPILOGUES)
def test_every_epilogue(epi):
    base.linear_case(torch.bfloat16, [1500, 0, 700], 1031, 1032, epi)
    base.linear_case(torch.float16, [260, 300], 2049, 1031, epi)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("counts,N,K", SHAPES)
def test_gradients(dt, f32, counts, N, K):
    base.test_product_gradients(dt, f32, counts, N, K)


@pytest.mark.parametrize("offset", [1, 2, 4])
@pytest.mark.parametrize("counts,N,K", [([2000], 1032, 1024), ([700, 900], 1031, 1025)])
def test_operands_off_a_16_byte_address(offset, counts, N, K):
    base.linear_case(torch.bfloat16, counts, N, K, base.EPILOGUES[4], offset=offset)
    m, dt = base._m(), torch.float16
    off, dev = base.table(counts)
    R, E = off[-1], len(counts)
    x, w, dy = (base.rand(s, dt, i, sg, offset) for i, (s, sg) in
                enumerate((((R, K), 1.0), ((E, N, K), K ** -0.5), ((R, N), 1.0))))
    dx, dw = m.moe_linear_grad(dy, x, w, dev)
    for e, (a, b) in enumerate(spans(off)):
        d, xx = dy[a:b].to(F64), x[a:b].to(F64)
        want = d @ w[e].to(F64)
        check("dx", dx[a:b], want, product_bound(N, d.abs() @ w[e].to(F64).abs()) + rounded(want, dt))
        want = d.t() @ xx
        check("dw", dw[e], want, product_bound(b - a, d.abs().t() @ xx.abs()) + rounded(want, dt))


@pytest.mark.parametrize("N,K", [(515, 1025), (512, 1031), (515, 1032)])
def test_neighbours_stay_out(N, K):
    """Expert 1's rows and weights are NaN: what lies behind the last row of an expert, and behind the end of
    each row in the next one, leaves the others' results as they are."""
    m, dt = base._m(), torch.bfloat16
    off, dev = base.table([900, 64, 700])
    R, E = off[-1], 3
    x, w, dy = base.rand((R, K), dt, 1), base.rand((E, N, K), dt, 2, 0.05), base.rand((R, N), dt, 3)
    clean = [m.moe_linear(x, w, dev), *m.moe_linear_grad(dy, x, w, dev)]
    bad_x, bad_w, bad_dy = x.clone(), w.clone(), dy.clone()
    bad_x[off[1]:off[2]] = float("nan")
    bad_dy[off[1]:off[2]] = float("inf")
    bad_w[1] = float("nan")
    got = [m.moe_linear(bad_x, bad_w, dev), *m.moe_linear_grad(bad_dy, bad_x, bad_w, dev)]
    keep = torch.ones(R, dtype=torch.bool, device="cuda")
    keep[off[1]:off[2]] = False
    for a, b in zip(clean[:2], got[:2]):
        assert torch.equal(a[keep], b[keep])
    assert torch.equal(clean[2][[0, 2]], got[2][[0, 2]])


@pytest.mark.parametrize("counts,N,K", [([1500, 0, 700], 1031, 2049), ([512], 513, 6145), ([2048], 2047, 1024)])
def test_captured(counts, N, K):
    """Replays see the operands' current values: the copies are made in every one."""
    m, dt = base._m(), torch.bfloat16
    off, dev = base.table(counts)
    R, E = off[-1], len(counts)
    x, w, dy = base.rand((R, K), dt, 1), base.rand((E, N, K), dt, 2, K ** -0.5), base.rand((R, N), dt, 3)

    def work():
        return [m.moe_linear(x, w, dev, activation="silu"), *m.moe_linear_grad(dy, x, w, dev)]
    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work()
    for step in range(3):
        for t, s in ((x, 1.0), (w, K ** -0.5), (dy, 1.0)):
            t.copy_(base.rand(t.shape, dt, 10 * step + 7, s))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, work()):
            assert torch.equal(a, b)


def test_output_may_be_the_gate_or_the_residual():
    m, dt = base._m(), torch.float16
    x, w = base.rand((700, 1025), dt, 1), base.rand((1, 1031, 1025), dt, 2, 0.03)
    mul, res = base.rand((700, 1031), dt, 3), base.rand((700, 1031), dt, 4)
    want = m.moe_linear(x, w, mul=mul, residual=res)
    for which in (mul, res):
        args = dict(mul=mul.clone(), residual=res.clone())
        args["mul" if which is mul else "residual"] = out = which.clone()
        assert torch.equal(m.moe_linear(x, w, out=out, **args), want)


def test_results_repeat_bit_for_bit():
    m, dt = base._m(), torch.bfloat16
    off, dev = base.table([1500, 0, 700])
    x, w, dy = base.rand((2200, 2049), dt, 1), base.rand((3, 1031, 2049), dt, 2), base.rand((2200, 1031), dt, 3)
    a = [m.moe_linear(x, w, dev), *m.moe_linear_grad(dy, x, w, dev)]
    b = [m.moe_linear(x, w, dev), *m.moe_linear_grad(dy, x, w, dev)]
    for p, q in zip(a, b):
        assert torch.equal(p, q)
