"""Host-side refusals of the 16-bit MoE operators (no GPU needed): bad
arguments are rejected before the device is touched, by the C ABI (with
pointers that are never dereferenced) and by the torch binding."""
import ctypes as C

import pytest
import torch

NULL, SHAPE, ALIGN, WORKSPACE, ARG = 1, 2, 3, 5, 6
FAKE, ODD = C.c_void_p(0x10000), C.c_void_p(0x10001)


@pytest.fixture(scope="module")
def L():
    from extreme_quantized_moe_amd import _lib
    return _lib


@pytest.fixture(scope="module")
def m():
    import extreme_quantized_moe_amd
    return extreme_quantized_moe_amd


@pytest.mark.parametrize("change,code", [
    (dict(x=None), NULL), (dict(pos=None), NULL), (dict(y=None), NULL), (dict(T=-1), SHAPE),
    (dict(T=(1 << 24) + 1), SHAPE), (dict(slots=0), SHAPE), (dict(slots=17), SHAPE), (dict(H=0), SHAPE),
    (dict(H=(1 << 20) + 1), SHAPE), (dict(rows=-1), SHAPE), (dict(rows=(1 << 28) + 1), SHAPE),
    (dict(dtype=3), ARG), (dict(dtype=-1), ARG), (dict(x=ODD), ALIGN), (dict(y=ODD), ALIGN), (dict(pos=ODD), ALIGN),
])
def test_dispatch_refusals(L, change, code):
    a = dict(x=FAKE, pos=FAKE, T=4, slots=2, H=64, rows=8, dtype=L.F16, y=FAKE)
    a.update(change)
    lib, tail = L.lib(), (a["T"], a["slots"], a["H"], a["rows"], a["dtype"])
    assert lib.milo_moe_permute(a["x"], a["pos"], *tail, a["y"], None) == code
    assert lib.milo_moe_permute_grad(a["y"], a["pos"], *tail, a["x"], None) == code
    assert lib.milo_moe_unpermute(a["y"], a["pos"], FAKE, *tail, a["x"], None) == code
    assert lib.milo_moe_unpermute_grad(a["x"], a["y"], a["pos"], FAKE, *tail, FAKE, FAKE, None) == code
    assert len(lib.milo_last_error()) > 0


def test_dispatch_refuses_missing_gradient_and_misaligned_weights(L):
    lib = L.lib()
    assert lib.milo_moe_unpermute_grad(FAKE, FAKE, FAKE, FAKE, 4, 2, 64, 8, L.F16, None, FAKE, None) == NULL
    assert lib.milo_moe_unpermute_grad(FAKE, FAKE, FAKE, ODD, 4, 2, 64, 8, L.F16, FAKE, FAKE, None) == ALIGN
    assert lib.milo_moe_unpermute(FAKE, FAKE, ODD, 4, 2, 64, 8, L.F16, FAKE, None) == ALIGN
    assert lib.milo_moe_unpermute(FAKE, FAKE, None, 4, 2, 64, 8, L.F32, C.c_void_p(0x10002), None) == ALIGN


def test_nothing_to_do_touches_nothing(L):
    lib = L.lib()
    assert lib.milo_moe_permute(None, None, 0, 2, 64, 0, L.F16, None, None) == 0
    assert lib.milo_moe_unpermute(None, None, None, 0, 2, 64, 0, L.F16, None, None) == 0
    assert lib.milo_moe_unpermute_grad(None, None, None, None, 0, 2, 64, 0, L.F16, None, None, None) == 0
    assert lib.milo_route_grad(None, None, None, 0, 8, 2, 0, 1, None, None) == 0
    assert lib.milo_moe_linear(C.byref(linear_desc(L, num_rows=0, x=None, y=None)), None, 0, None) == 0


@pytest.mark.parametrize("T,E,k,S", [(-1, 8, 2, 0), (1 << 25, 8, 2, 0), (4, 0, 1, 0), (4, 8, 0, 0), (4, 8, 9, 0),
                                     (4, 2, 3, 0), (4, 255, 2, 2), (4, 16, 8, 9), (4, 8, 2, -1)])
def test_route_grad_shapes(L, T, E, k, S):
    assert L.lib().milo_route_grad(FAKE, FAKE, FAKE, T, E, k, S, 1, FAKE, None) == SHAPE


def test_route_grad_pointers(L):
    lib = L.lib()
    for i in range(4):
        p = [FAKE] * 4
        p[i] = None
        assert lib.milo_route_grad(p[0], p[1], p[2], 4, 8, 2, 0, 1, p[3], None) == NULL
        p[i] = ODD
        assert lib.milo_route_grad(p[0], p[1], p[2], 4, 8, 2, 0, 1, p[3], None) == ALIGN


def linear_desc(L, **kw):
    d = L.MiloLinearDesc()
    d.num_experts, d.N, d.K, d.num_rows = 4, 64, 128, 32
    d.dtype = d.out_dtype = L.BF16
    d.x = d.w = d.offsets = d.y = 0x10000
    for k, v in kw.items():
        setattr(d, k, v)
    return d


LINEAR_BAD = [
    (dict(num_experts=0), SHAPE), (dict(num_experts=257), SHAPE), (dict(N=0), SHAPE), (dict(N=65537), SHAPE),
    (dict(K=0), SHAPE), (dict(K=65537), SHAPE), (dict(num_rows=-1), SHAPE), (dict(num_rows=(1 << 20) + 1), SHAPE),
    (dict(offsets=None), NULL), (dict(offsets=0x10002), ALIGN), (dict(dtype=2), ARG), (dict(w=0x10001), ALIGN),
    (dict(x=0x10001), ALIGN),
]


@pytest.mark.parametrize("change,code", LINEAR_BAD + [
    (dict(x=None), NULL), (dict(w=None), NULL), (dict(y=None), NULL), (dict(out_dtype=0), ARG),
    (dict(out_dtype=3), ARG), (dict(activation=5), ARG), (dict(activation=-1), ARG),
    (dict(max_rows_per_expert=-1), SHAPE), (dict(bias=0x10001), ALIGN), (dict(mul=0x10001), ALIGN),
    (dict(residual=0x10001), ALIGN), (dict(pre=0x10001), ALIGN), (dict(y=0x10002, out_dtype=2), ALIGN),
])
def test_linear_refusals(L, change, code):
    assert L.lib().milo_moe_linear(C.byref(linear_desc(L, **change)), None, 0, None) == code
    assert L.lib().milo_moe_linear_workspace_bytes(C.byref(linear_desc(L, **change))) == 0


def grad_desc(L, **kw):
    d = L.MiloLinearGradDesc()
    d.num_experts, d.N, d.K, d.num_rows = 4, 64, 128, 32
    d.dtype = d.dw_dtype = L.BF16
    d.dy = d.x = d.w = d.offsets = d.dx = d.dw = 0x10000
    for k, v in kw.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("change,code", LINEAR_BAD + [
    (dict(dy=None), NULL), (dict(x=None), NULL), (dict(w=None), NULL), (dict(dw_dtype=0), ARG),
    (dict(dy=0x10001), ALIGN), (dict(dx=0x10001), ALIGN), (dict(dw=0x10001), ALIGN),
    (dict(dw=0x10002, dw_dtype=2), ALIGN), (dict(dx_add=0x10001), ALIGN),
])
def test_linear_grad_refusals(L, change, code):
    assert L.lib().milo_moe_linear_grad(C.byref(grad_desc(L, **change)), None, 0, None) == code


def act_grad_args(L, **kw):
    a = dict(dy=FAKE, pre=FAKE, mul=None, offsets=FAKE, E=4, N=64, rows=32, dtype=L.F16, act=L.ACT_SILU, dpre=FAKE,
             dmul=None, dbias=None, ws=None, nbytes=0)
    a.update(kw)
    return (*a.values(), None)


@pytest.mark.parametrize("change,code", [
    (dict(dy=None), NULL), (dict(pre=None), NULL), (dict(dpre=None), NULL), (dict(mul=FAKE), ARG),
    (dict(dmul=FAKE), ARG), (dict(dtype=2), ARG), (dict(act=5), ARG), (dict(E=0), SHAPE), (dict(E=257), SHAPE),
    (dict(N=0), SHAPE), (dict(rows=-1), SHAPE), (dict(offsets=None), NULL), (dict(dbias=FAKE), WORKSPACE),
    (dict(dbias=FAKE, ws=FAKE, nbytes=256), WORKSPACE), (dict(dbias=FAKE, ws=C.c_void_p(0x10010), nbytes=1 << 20), ALIGN),
    (dict(dbias=C.c_void_p(0x10002), ws=FAKE, nbytes=1 << 20), ALIGN), (dict(dy=ODD), ALIGN), (dict(dpre=ODD), ALIGN),
])
def test_act_grad_refusals(L, change, code):
    assert L.lib().milo_moe_linear_act_grad(*act_grad_args(L, **change)) == code


def test_null_descriptors(L):
    lib = L.lib()
    assert lib.milo_moe_linear(None, None, 0, None) == NULL
    assert lib.milo_moe_linear_grad(None, None, 0, None) == NULL


# ------------------------------------------------------------------ binding

def test_binding_refuses_host_tensors(m):
    x = torch.zeros((4, 64), dtype=torch.float16)
    pos = torch.zeros(8, dtype=torch.int32)
    w = torch.zeros((32, 64), dtype=torch.float16)
    dy = torch.zeros((4, 32), dtype=torch.float16)
    for call in (lambda: m.moe_permute(x, pos, 2), lambda: m.moe_unpermute(x, pos, 2),
                 lambda: m.moe_unpermute_grad(x, x, pos, 2), lambda: m.moe_linear(x, w),
                 lambda: m.moe_linear_grad(dy, x, w), lambda: m.moe_linear_act_grad(dy, dy, "silu"),
                 lambda: m.route_grad(torch.zeros(8), torch.zeros((4, 8)), torch.zeros((4, 2), dtype=torch.int32))):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_binding_refuses_types_and_ranks(m):
    with pytest.raises(ValueError, match="unsupported type"):
        m.moe_permute(torch.zeros((4, 64), dtype=torch.float64), torch.zeros(8, dtype=torch.int32), 2)
    with pytest.raises(ValueError, match="unsupported type"):
        m.moe_linear(torch.zeros((4, 64)), torch.zeros((8, 64)))
    with pytest.raises(ValueError, match=r"\[T\]\[H\]"):
        m.moe_permute(torch.zeros(64, dtype=torch.float16), torch.zeros(8, dtype=torch.int32), 2)
    with pytest.raises(ValueError, match="w1 and w3"):
        m.MoELayer16(torch.zeros((2, 8, 4)), torch.zeros((2, 8, 5)), torch.zeros((2, 4, 8)), 2, 1)
