"""Buffers that the header lets two operands share, through the C ABI: the
activation gradient written over its inputs, the input gradient over the
gradient added to it.  Results are those of separate buffers, bit for bit."""
import ctypes as C
import itertools

import pytest
import torch

from tests.test_gpu_linear import rand, table

pytestmark = pytest.mark.gpu


def _lib():
    from extreme_quantized_moe_amd import _lib
    return _lib


def stream():
    return C.c_void_p(torch.cuda.current_stream().cuda_stream)


def act_grad(dy, pre, mul, dev, E, dpre, dmul, bias):
    L = _lib()
    R, N = dy.shape
    db = torch.empty((E, N), device="cuda") if bias else None
    nbytes = L.lib().milo_moe_linear_act_grad_workspace_bytes(E, N, R) if bias else 0
    ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device="cuda")
    p = [None if t is None else t.data_ptr() for t in (dy, pre, mul, dev, dpre, dmul, db)]
    dt = L.F16 if dy.dtype == torch.float16 else L.BF16
    rc = L.lib().milo_moe_linear_act_grad(*p[:4], E, N, R, dt, L.ACT_GELU, *p[4:], ws.data_ptr(), nbytes, stream())
    assert rc == 0, L.lib().milo_last_error()
    return db


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("counts,N", [([5], 8), ([40, 0, 70], 264), ([1, 33, 2], 61), ([1100, 3], 1030), ([300, 500], 2048)])
def test_activation_gradient_over_its_inputs(dt, bias, counts, N):
    off, dev = table(counts)
    R, E = off[-1], len(counts)
    src = [rand((R, N), dt, i, s) for i, s in ((1, 1.0), (2, 2.0), (3, 1.0))]
    dpre, dmul = torch.empty_like(src[0]), torch.empty_like(src[0])
    db = act_grad(*src, dev, E, dpre, dmul, bias)
    alone = torch.empty_like(src[0])
    db_alone = act_grad(src[0], src[1], None, dev, E, alone, None, bias)
    for a, b in itertools.permutations(range(4), 2):        # 3: a buffer of its own
        own = [t.clone() for t in src] + [torch.empty_like(src[0])]
        got = act_grad(*own[:3], dev, E, own[a], own[b], bias)
        assert torch.equal(own[a], dpre) and torch.equal(own[b], dmul), (a, b)
        assert not bias or torch.equal(got, db)
    for a in range(2):
        own = [t.clone() for t in src[:2]]
        got = act_grad(*own, None, dev, E, own[a], None, bias)
        assert torch.equal(own[a], alone) and (not bias or torch.equal(got, db_alone))


@pytest.mark.parametrize("counts,N,K", [([9, 0, 3], 512, 1024), ([100], 4096, 384), ([900, 40, 0, 800], 512, 2048),
                                        ([150, 3], 131, 1031), ([2048], 2047, 1024), ([640], 2050, 2046)])
def test_input_gradient_over_what_is_added(counts, N, K):
    """The split, tile, register-staged and copying forms of dx."""
    L, dt = _lib(), torch.bfloat16
    off, dev = table(counts)
    R, E = off[-1], len(counts)
    dy, w, add = rand((R, N), dt, 1), rand((E, N, K), dt, 2, N ** -0.5), rand((R, K), dt, 3)

    def run(dx_add, dx):
        d = L.MiloLinearGradDesc(E, N, K, R, L.BF16, L.BF16, dy.data_ptr(), None, w.data_ptr(), dev.data_ptr(),
                                 dx_add.data_ptr(), dx.data_ptr(), None)
        nbytes = L.lib().milo_moe_linear_grad_workspace_bytes(C.byref(d))
        ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device="cuda")
        assert L.lib().milo_moe_linear_grad(C.byref(d), ws.data_ptr(), nbytes, stream()) == 0
        return dx

    want = run(add, torch.empty_like(add))
    own = add.clone()
    assert torch.equal(run(own, own), want)
