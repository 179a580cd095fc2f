"""Rows to the experts and back, and their gradients, on the GPU against
float64 definitions: types, odd widths, misaligned buffers, dropped pairs,
positions out of range, free rows left as they were, non-finite values next to
masked pairs, more bytes than 32 bits address."""
import pytest
import torch

from tests.moe16_reference import F64, U32, check, rounded

pytestmark = pytest.mark.gpu
TYPES = [torch.float16, torch.bfloat16, torch.float32]


def _m():
    import extreme_quantized_moe_amd as m
    return m


def table(T, slots, dropped, free, seed):
    """(pos [T*slots], num_rows): a random placement with `dropped` pairs left out and `free` rows unused."""
    g = torch.Generator().manual_seed(seed)
    P = T * slots
    kept = P - dropped
    rows = kept + free
    pos = torch.full((P,), -1, dtype=torch.int32)
    who = torch.randperm(P, generator=g)[:kept]
    pos[who] = torch.randperm(rows, generator=g)[:kept].to(torch.int32)
    return pos, rows


def rand(shape, dt, seed, offset=0):
    """Normal values; offset > 0 puts the tensor that many elements behind an aligned address."""
    g = torch.Generator().manual_seed(seed)
    n = 1
    for s in shape:
        n *= s
    v = torch.randn(n + offset, generator=g).to(dt).cuda()
    return v[offset:].view(shape)


CASES = [  # T, slots, H, dropped, free
    (1, 1, 1, 0, 0), (1, 2, 8, 1, 0), (1, 8, 4096, 0, 0), (3, 2, 7, 2, 3), (5, 3, 33, 4, 1), (16, 2, 4096, 0, 0),
    (17, 8, 264, 9, 5), (40, 16, 130, 100, 0), (64, 5, 65, 0, 2), (2, 2, 9, 4, 3), (130, 4, 2048, 7, 1),
    (2100, 2, 520, 30, 0), (2, 1, 6000, 0, 0), (7, 9, 1032, 5, 5),
]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,slots,H,dropped,free", CASES)
def test_there_and_back(dt, T, slots, H, dropped, free):
    m = _m()
    pos, rows = table(T, slots, dropped, free, T * 31 + H)
    P = T * slots
    x = rand((T, H), dt, 1)
    y = rand((rows, H), dt, 2) if rows else torch.zeros((0, H), dtype=dt, device="cuda")
    w = rand((P,), torch.float32, 3)
    dev = pos.cuda()
    ys = m.moe_permute(x, dev, slots, num_rows=rows, out=torch.full((rows, H), 7.0, dtype=dt, device="cuda"))
    want = torch.full((rows, H), 7.0, dtype=dt)
    xc = x.cpu()
    for p in range(P):
        if pos[p] >= 0:
            want[pos[p]] = xc[p // slots]
    assert torch.equal(ys.cpu(), want)
    yc, wc = y.cpu().to(F64), w.cpu().to(F64)
    at = pos.clamp(min=0).long()
    kept = (pos >= 0).to(F64)
    rowsum = torch.zeros((T, slots, H), dtype=F64) if rows == 0 else (yc[at] * kept[:, None]).view(T, slots, H)
    weighted = rowsum * wc.view(T, slots, 1)
    for got, terms in ((m.moe_unpermute(y, dev, slots, w), weighted), (m.moe_unpermute(y, dev, slots), rowsum),
                       (m.moe_permute_grad(y, dev, slots), rowsum)):
        check("sum", got.cpu(), terms.sum(1), rounded(terms.sum(1), dt) + 2 * slots * U32 * terms.abs().sum(1))


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("T,slots,H,dropped,free", CASES)
def test_unpermute_grad(dt, weighted, T, slots, H, dropped, free):
    m = _m()
    pos, rows = table(T, slots, dropped, free, T * 37 + H)
    P = T * slots
    dout, y = rand((T, H), dt, 4), rand((rows, H), dt, 5)
    w = rand((P,), torch.float32, 6) if weighted else None
    dy, dw = m.moe_unpermute_grad(dout, y, pos.cuda(), slots, w,
                                  out=torch.full((rows, H), 7.0, dtype=dt, device="cuda"))
    d, yc = dout.cpu().to(F64), y.cpu().to(F64)
    want_dy = torch.full((rows, H), 7.0, dtype=F64)
    want_dw = torch.zeros(P, dtype=F64)
    mag = torch.zeros(P, dtype=F64)
    for p in range(P):
        if pos[p] >= 0:
            want_dy[pos[p]] = d[p // slots] * (float(w[p]) if weighted else 1.0)
            want_dw[p] = (d[p // slots] * yc[pos[p]]).sum()
            mag[p] = (d[p // slots] * yc[pos[p]]).abs().sum()
    check("dy", dy.cpu(), want_dy, rounded(want_dy, dt) + U32 * want_dy.abs())
    check("dw", dw.cpu(), want_dw, (H + 2) * U32 * mag + 1e-30)
    assert torch.equal(dw.cpu()[pos < 0], torch.zeros(int((pos < 0).sum())))


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("offset", [1, 2, 4])
def test_misaligned_buffers(dt, offset):
    """Rows of a 16-byte multiple in buffers that start off a 16-byte address."""
    m = _m()
    pos, rows = table(33, 3, 5, 2, 9)
    x, y, w = rand((33, 64), dt, 1, offset), rand((rows, 64), dt, 2, offset), rand((99,), torch.float32, 3)
    p = pos.cuda()
    assert torch.equal(m.moe_permute(x, p, 3, num_rows=rows, dropped=True),
                       m.moe_permute(x.clone(), p, 3, num_rows=rows, dropped=True))
    assert torch.equal(m.moe_unpermute(y, p, 3, w), m.moe_unpermute(y.clone(), p, 3, w))
    a, b = m.moe_unpermute_grad(x, y, p, 3, w, dropped=True), m.moe_unpermute_grad(x.clone(), y.clone(), p, 3, w,
                                                                                   dropped=True)
    assert torch.equal(a[0], b[0])
    check("dw", a[1].cpu(), b[1].cpu().to(F64), torch.full((99,), 64 * 64 * U32, dtype=F64))


def test_masked_pairs_add_nothing_whatever_they_hold():
    """A dropped pair's weight may be NaN or infinite, free rows too; a token without a pair gets zeros."""
    m = _m()
    dt, T, slots, H = torch.bfloat16, 4, 3, 72
    pos = torch.tensor([0, -1, 1, -1, -1, -1, 2, 99, -2147483648, 4, 2147483647, 5], dtype=torch.int32)
    y = rand((6, H), dt, 2)
    y[3] = float("nan")
    w = rand((12,), torch.float32, 3)
    w[pos.cuda() < 0] = float("nan")
    w[7], w[10] = float("inf"), float("-inf")
    out = m.moe_unpermute(y, pos.cuda(), slots, w)
    assert torch.isfinite(out.float()).all() and torch.equal(out[1], torch.zeros_like(out[1]))
    dout = rand((T, H), dt, 4)
    dy, dw = m.moe_unpermute_grad(dout, y, pos.cuda(), slots, w, dropped=True)
    assert torch.isfinite(dy.float()).all() and torch.equal(dy[3], torch.zeros_like(dy[3]))
    masked = ((pos < 0) | (pos >= 6)).cuda()
    assert torch.equal(dw[masked], torch.zeros_like(dw[masked])) and torch.isfinite(dw).all()
    x = rand((T, H), dt, 5)
    ys = m.moe_permute(x, pos.cuda(), slots, num_rows=6, dropped=True)
    assert torch.equal(ys[0], x[0]) and torch.equal(ys[3], torch.zeros_like(ys[3])) and torch.equal(ys[5], x[3])


def test_every_pair_dropped_and_no_rows():
    m = _m()
    pos = torch.full((6,), -1, dtype=torch.int32, device="cuda")
    empty = torch.zeros((0, 40), dtype=torch.float16, device="cuda")
    x = rand((3, 40), torch.float16, 1)
    assert m.moe_permute(x, pos, 2, num_rows=0).shape == (0, 40)
    assert torch.equal(m.moe_unpermute(empty, pos, 2), torch.zeros_like(x))
    dy, dw = m.moe_unpermute_grad(x, empty, pos, 2)
    assert dy.shape == (0, 40) and torch.equal(dw, torch.zeros(6, device="cuda"))
    none = torch.zeros((0,), dtype=torch.int32, device="cuda")
    assert m.moe_permute(empty, none, 2).shape == (0, 40)


def test_rows_behind_32_bits():
    """An expert-ordered buffer of 5 GiB: its last rows are reached."""
    m = _m()
    H, rows = 1 << 16, 40000
    y = torch.zeros((rows, H), dtype=torch.bfloat16, device="cuda")
    pos = torch.tensor([rows - 1, 0, rows - 2, 20000], dtype=torch.int32, device="cuda")
    x = rand((2, H), torch.bfloat16, 1)
    m.moe_permute(x, pos, 2, out=y)
    assert torch.equal(y[rows - 1], x[0]) and torch.equal(y[rows - 2], x[1]) and torch.equal(y[20000], x[1])
    assert torch.equal(m.moe_permute_grad(y, pos, 2), (2 * x.float()).to(torch.bfloat16))


@pytest.mark.parametrize("E,k,S,renorm", [(8, 2, 0, True), (64, 6, 2, False), (5, 5, 1, True), (1, 1, 0, False),
                                          (256, 8, 0, False), (200, 8, 8, True), (65, 1, 0, True)])
@pytest.mark.parametrize("T", [1, 3, 130])
def test_route_grad(E, k, S, renorm, T):
    m = _m()
    g = torch.Generator().manual_seed(E + T)
    logits = torch.randn((T, E), generator=g) * 2
    if E > 8:
        logits[0, 0] = torch.finfo(torch.float32).min     # an expert that a mask rules out
    r = m.route_sort(logits.cuda(), k, S, renorm)
    gw = torch.randn((T * (k + S),), generator=g)
    got = m.route_grad(gw.cuda(), logits.cuda(), r["ids"], S, renorm).cpu()
    l = logits.to(F64).requires_grad_(True)
    ids = r["ids"].cpu().long()
    p = torch.softmax(l.gather(1, ids), 1) if renorm else torch.softmax(l, 1).gather(1, ids)
    (p * gw.view(T, k + S)[:, :k].to(F64)).sum().backward()
    # float32: exp of differences up to ~20 (20 roundings), sums over E, a difference of terms up to max |g|
    bound = (E + 40) * U32 * gw.abs().max().to(F64) * torch.ones_like(l)
    check("dlogits", got, l.grad, bound)
    # central differences of the routed weights along a random direction, picks held
    u = torch.randn((T, E), generator=g).to(F64)
    u[logits < -1e30] = 0

    def f(v):
        q = torch.softmax(v.gather(1, ids), 1) if renorm else torch.softmax(v, 1).gather(1, ids)
        return float((q * gw.view(T, k + S)[:, :k].to(F64)).sum())
    h = 1e-5
    diff = (f(logits.to(F64) + h * u) - f(logits.to(F64) - h * u)) / (2 * h)
    assert abs(diff - float((got.to(F64) * u).sum())) <= float((bound * u.abs()).sum()) + 1e-6 * T
