"""Rows of a new expert-ordered tensor that no pair names are zeros, whatever
the memory held before; rows of a buffer that is handed over stay."""
import ctypes as C

import pytest
import torch

NULL, SHAPE = 1, 2
FAKE = C.c_void_p(0x10000)


def _m():
    import extreme_quantized_moe_amd as m
    return m


def test_zeroed_forms_refuse_missing_buffers():
    L = _m()._lib
    lib = L.lib()
    tail = (0, 2, 64, 8, L.F16)
    assert lib.milo_moe_permute_zeroed(None, None, *tail, None, None) == NULL
    assert lib.milo_moe_unpermute_grad_zeroed(None, FAKE, None, None, *tail, None, None, None) == NULL
    assert lib.milo_moe_permute_zeroed(FAKE, FAKE, 4, 0, 64, 8, L.F16, FAKE, None) == SHAPE
    assert lib.milo_moe_permute_zeroed(None, None, 0, 2, 64, 0, L.F16, None, None) == 0      # nothing to write


def dirty(shape, dt):
    """NaN in the memory that the next tensor of this size takes."""
    t = torch.full(shape, float("nan"), dtype=dt, device="cuda")
    del t


def table(T, slots, kept, rows, seed):
    g = torch.Generator().manual_seed(seed)
    pos = torch.randint(-3, 0, (T * slots,), generator=g, dtype=torch.int32)
    pos[torch.randperm(T * slots, generator=g)[:1]] = 2 ** 31 - 1 if kept < T * slots else -1
    who = torch.randperm(T * slots, generator=g)[:kept]
    pos[who] = torch.randperm(rows, generator=g)[:kept].to(torch.int32)
    return pos.cuda()


CASES = [  # T, slots, H, pairs kept, rows
    (1, 1, 1, 0, 1), (1, 1, 8, 1, 1), (5, 3, 33, 11, 15), (16, 2, 4096, 20, 32), (16, 2, 264, 32, 31 + 32), (40, 2, 7, 64, 129),
    (700, 3, 131, 1500, 2100), (4096, 2, 72, 8192, 8192), (4096, 2, 64, 6000, 4 * 4097), (9000, 8, 8, 60000, 72000),
    (30000, 9, 8, 200000, 270000), (30000, 9, 3, 100001, 100001), (3, 2, 16, 5, 4200000),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,slots,H,kept,rows", CASES)
def test_rows_without_a_pair_are_zeros(dt, T, slots, H, kept, rows):
    m = _m()
    pos = table(T, slots, kept, rows, T + H)
    x = torch.randn((T, H), device="cuda").to(dt)
    held = torch.full((rows, H), 7.0, dtype=dt, device="cuda")
    named = torch.zeros(rows, dtype=torch.bool, device="cuda")
    ok = (pos >= 0) & (pos < rows)
    named[pos[ok].long()] = True
    assert int(named.sum()) == kept
    m.moe_permute(x, pos, slots, out=held)
    assert bool((held[~named] == 7).all())
    want = torch.where(named[:, None], held, torch.zeros_like(held))
    dirty((rows, H), dt)
    assert torch.equal(m.moe_permute(x, pos, slots, num_rows=rows), want)
    y = torch.randn((rows, H), device="cuda").to(dt)
    w = torch.randn(T * slots, device="cuda")
    held = torch.full((rows, H), 7.0, dtype=dt, device="cuda")
    _, dw = m.moe_unpermute_grad(x, y, pos, slots, w, out=held)
    want = torch.where(named[:, None], held, torch.zeros_like(held))
    dirty((rows, H), dt)
    dy, dw2 = m.moe_unpermute_grad(x, y, pos, slots, w)
    assert torch.equal(dy, want) and torch.equal(dw, dw2)


@pytest.mark.gpu
def test_default_row_count_with_dropped_pairs():
    m = _m()
    x = torch.randn((6, 40), device="cuda").half()
    pos = torch.tensor([0, -1, 1, -1, 2, -1, 3, -1, 4, -1, 5, 11], dtype=torch.int32, device="cuda")
    dirty((12, 40), torch.float16)
    y = m.moe_permute(x, pos, 2)
    assert torch.equal(y[:6], x) and torch.equal(y[11], x[5]) and torch.equal(y[6:11], torch.zeros_like(y[6:11]))


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.float16, torch.float32])
def test_no_token(dt):
    m = _m()
    pos = torch.zeros(0, dtype=torch.int32, device="cuda")
    x = torch.zeros((0, 33), dtype=dt, device="cuda")
    dirty((70, 33), dt)
    y = m.moe_permute(x, pos, 2, num_rows=70)
    assert y.shape == (70, 33) and not y.any()
    dirty((70, 33), dt)
    dy, dw = m.moe_unpermute_grad(x, y, pos, 2)
    assert not dy.any() and dw.numel() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("offset,rows,H", [(0, 5, 7), (1, 5, 7), (1, 1, 1), (0, 1, 1), (1, 1, 2), (3, 1000, 1111)])
def test_only_the_rows_are_written(offset, rows, H):
    """A buffer off a 4-byte address, with an odd number of values, no token."""
    L = _m()._lib
    n = rows * H
    buf = torch.full((offset + n + 5,), 7.0, dtype=torch.bfloat16, device="cuda")
    stream = C.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert L.lib().milo_moe_permute_zeroed(None, None, 0, 2, H, rows, L.BF16, buf.data_ptr() + 2 * offset, stream) == 0
    assert not buf[offset:offset + n].any()
    assert bool((buf[:offset] == 7).all()) and bool((buf[offset + n:] == 7).all())


@pytest.mark.gpu
def test_captured():
    m = _m()
    T, slots, H = 64, 2, 264
    x, pos = torch.randn((T, H), device="cuda").half(), table(T, slots, 100, 128, 1)
    m.moe_permute(x, pos, slots)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = m.moe_permute(x, pos, slots)
        dy, dw = m.moe_unpermute_grad(x, y, pos, slots)
    for i in range(4):
        x.copy_(torch.randn((T, H), device="cuda").half())
        pos.copy_(table(T, slots, 20 * i, 128, 50 + i))
        g.replay()
        torch.cuda.synchronize()
        want = m.moe_permute(x, pos, slots)
        dirty((128, H), torch.float16)
        want_dy, want_dw = m.moe_unpermute_grad(x, want, pos, slots)
        assert torch.equal(y, want) and torch.equal(dy, want_dy) and torch.equal(dw, want_dw)
        assert int((~y.any(1)).sum()) >= 128 - 20 * i


@pytest.mark.gpu
def test_more_rows_than_pairs_are_zeros_whatever_the_caller_says():
    m = _m()
    x = torch.randn((6, 40), device="cuda").half()
    pos = torch.arange(12, dtype=torch.int32, device="cuda")
    for dropped in (None, False, True):
        dirty((20, 40), torch.float16)
        y = m.moe_permute(x, pos, 2, num_rows=20, dropped=dropped)
        assert torch.equal(y[:12], x.repeat_interleave(2, 0)) and not y[12:].any()
        dy, _ = m.moe_unpermute_grad(x, y, pos, 2, dropped=dropped)
        assert torch.equal(dy, y)
    assert torch.equal(m.moe_permute(x, pos, 2, dropped=False), y[:12])
