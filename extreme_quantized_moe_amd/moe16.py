"""torch-facing binding of the 16-bit MoE operators (include/milo.h): rows to
the experts and back, grouped products with an epilogue, their gradients, and
`MoELayer16`, the unquantized counterpart of `MoELayer` with a backward pass.
Calls run on the tensors' device, on its current stream, and allocate their
outputs and scratch from torch's allocator; nothing is kept between calls.
They stand outside autograd: results carry no graph, also of operands that
require gradients, and the gradients are calls of their own."""
import ctypes as C

import torch

from . import _lib as L
from ._lib import check
from .ops import route_sort

_DTYPES = {torch.float16: L.F16, torch.bfloat16: L.BF16, torch.float32: L.F32}
_ACTS = {"none": L.ACT_NONE, "relu": L.ACT_RELU, "silu": L.ACT_SILU, "gelu": L.ACT_GELU,
         "gelu_tanh": L.ACT_GELU_TANH}


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _tensor(name, t, dtype, shape, dev=None):
    """Refuses a tensor the kernels could not address as they will."""
    if t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous() and (dev is None or t.device == dev):
        return
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: libmilo needs contiguous CUDA (HIP) tensors")
    raise ValueError(f"{name} is on {t.device}, the first operand on {dev}")


def _apart(out, *inputs, same=()):
    """Refuses an `out` that shares memory with an input: other threads would
    read what was just written.  same: inputs that may be `out` itself."""
    lo = out.data_ptr()
    hi = lo + out.numel() * out.element_size()
    for i, t in enumerate((*inputs, *same)):
        if t is None:
            continue
        a, n = t.data_ptr(), t.numel() * t.element_size()
        if a < hi and lo < a + n and (i < len(inputs) or a != lo or t.dtype != out.dtype):
            raise ValueError("out shares memory with an input")


def _float_type(name, t, wide=True):
    code = _DTYPES.get(t.dtype)
    if code is None or (code == L.F32 and not wide):
        raise ValueError(f"{name}: unsupported type {t.dtype}")
    return code


def _too_large(*sizes):
    """The library's sizes are 32-bit numbers, and ctypes would pass larger
    ones on modulo 2^32, as others that are allowed.  Callers test
    (a | b | ...) >> 31: true for a size outside 0 .. 2^31 - 1."""
    raise ValueError(f"a size does not fit a 32-bit number: {', '.join(map(str, sizes))}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _call(name, dev, *args):
    """The library's `name` with `dev` as the current device: launches go there,
    and plans (so workspace sizes too) take its number of compute units."""
    fn = getattr(L.lib(), name)
    if torch._C._cuda_getDevice() == dev.index:
        return fn(*args)
    with torch.cuda.device(dev):
        return fn(*args)


def _run(name, dev, *args):
    """Calls the library's `name` with (*args, stream) on the device's current
    stream.  (torch.cuda.current_stream builds a Stream object for this; a
    decoding step's calls take a few microseconds in all.)"""
    index = dev.index
    stream = torch._C._cuda_getCurrentRawStream(index)
    if torch._C._cuda_getDevice() == index:
        rc = getattr(L.lib(), name)(*args, stream)
    else:
        rc = _call(name, dev, *args, stream)
    if rc:
        check(name, rc)


def _scratch(nbytes, dev):
    """Scratch of one call: torch's allocator orders its reuse on the stream
    and keeps it apart for a captured graph."""
    return torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None


# ------------------------------------------------------------------ dispatch

def _pairs(pair_pos, slots, dev):
    n = pair_pos.numel()
    if n >> 31:
        _too_large(n)
    _need(slots >= 1 and n % slots == 0, f"pair_pos holds {n} entries, not a multiple of {slots} slots")
    _tensor("pair_pos", pair_pos, torch.int32, pair_pos.shape, dev)
    return n // slots


def _rows_out(name, num_rows, H, pairs, like, dropped):
    """A new expert-ordered output, and the call that writes every row of it:
    the _zeroed one unless the caller says that every row has a pair."""
    if num_rows >> 31:
        _too_large(num_rows)
    whole = dropped is not None and not dropped and num_rows <= pairs
    return name if whole else name + "_zeroed", torch.empty((num_rows, H), dtype=like.dtype, device=like.device)


def moe_permute(x, pair_pos, slots, num_rows=None, dropped=None, out=None):
    """Rows into expert order: y[pair_pos[t, j]] = x[t].  x [T][H] fp16, bf16
    or fp32; pair_pos int32 [T*slots] as from `route_sort`, negative for a
    dropped pair.  Returns y [num_rows][H] (default T*slots).  Rows that no
    pair names are zeros in a new tensor; those of `out` keep their values.
    dropped=False says that every one of at most T*slots rows has a pair, as with
    a table straight from `route_sort`: the rows are then not looked over (which
    takes some microseconds for many narrow ones), and one without a pair is
    uninitialised."""
    code = _float_type("x", x)
    _need(x.dim() == 2, "x must be [T][H]")
    dev = x.device
    T, H = x.shape
    if (T | H | slots) >> 31:
        _too_large(T, H, slots)
    _tensor("x", x, x.dtype, x.shape)
    _need(_pairs(pair_pos, slots, dev) == T, f"pair_pos must hold {T} x {slots} entries")
    if out is None:
        num_rows = T * slots if num_rows is None else num_rows
        name, out = _rows_out("milo_moe_permute", num_rows, H, T * slots, x, dropped)
    else:
        name = "milo_moe_permute"
        num_rows = out.shape[0] if num_rows is None else num_rows
        if num_rows >> 31:
            _too_large(num_rows)
        _tensor("out", out, x.dtype, (num_rows, H), dev)
        _apart(out, x, pair_pos)
    _run(name, dev, x.data_ptr(), pair_pos.data_ptr(), T, slots, H, num_rows, code, out.data_ptr())
    return out


def moe_permute_grad(dy, pair_pos, slots, out=None):
    """Gradient of `moe_permute`: dx[t] = sum of dy over the token's kept
    pairs (fp32, slot order, rounded once).  dy [num_rows][H]; returns [T][H]."""
    return moe_unpermute(dy, pair_pos, slots, None, out)


def moe_unpermute(y, pair_pos, slots, slot_w=None, out=None):
    """Rows back to their tokens: out[t] = sum over kept slots of
    slot_w[t, j] * y[pair_pos[t, j]] (fp32, slot order, rounded once; zeros
    without a kept pair).  y [num_rows][H]; slot_w fp32 [T*slots] or None
    (weights 1).  Returns [T][H]."""
    code = _float_type("y", y)
    _need(y.dim() == 2, "y must be [num_rows][H]")
    dev = y.device
    R, H = y.shape
    if (R | H | slots) >> 31:
        _too_large(R, H, slots)
    _tensor("y", y, y.dtype, y.shape)
    T = _pairs(pair_pos, slots, dev)
    if slot_w is not None:
        _tensor("slot_w", slot_w, torch.float32, pair_pos.shape, dev)
    if out is None:
        out = torch.empty((T, H), dtype=y.dtype, device=dev)
    else:
        _tensor("out", out, y.dtype, (T, H), dev)
        _apart(out, y, pair_pos, slot_w)
    _run("milo_moe_unpermute", dev, y.data_ptr(), pair_pos.data_ptr(), _ptr(slot_w), T, slots, H, R, code,
         out.data_ptr())
    return out


def moe_unpermute_grad(dout, y, pair_pos, slots, slot_w=None, dropped=None, out=None):
    """Gradients of `moe_unpermute`: (dy [num_rows][H], dslot_w fp32 [T*slots])
    with dy[pair_pos[t, j]] = slot_w[t, j] * dout[t] and dslot_w[t, j] =
    <dout[t], y[pair_pos[t, j]]>.  Rows of dy without a pair: as in
    `moe_permute`."""
    code = _float_type("dout", dout)
    _need(dout.dim() == 2 and y.dim() == 2, "dout must be [T][H] and y [num_rows][H]")
    dev = dout.device
    T, H = dout.shape
    R = y.shape[0]
    if (T | H | R | slots) >> 31:
        _too_large(T, H, R, slots)
    _tensor("dout", dout, dout.dtype, dout.shape)
    _tensor("y", y, dout.dtype, (R, H), dev)
    _need(_pairs(pair_pos, slots, dev) == T, f"pair_pos must hold {T} x {slots} entries")
    if slot_w is not None:
        _tensor("slot_w", slot_w, torch.float32, pair_pos.shape, dev)
    if out is None:
        name, out = _rows_out("milo_moe_unpermute_grad", R, H, T * slots, dout, dropped)
    else:
        name = "milo_moe_unpermute_grad"
        _tensor("out", out, dout.dtype, (R, H), dev)
        _apart(out, dout, y, pair_pos, slot_w)
    dw = torch.empty(pair_pos.shape, dtype=torch.float32, device=dev)
    _run(name, dev, dout.data_ptr(), y.data_ptr(), pair_pos.data_ptr(), _ptr(slot_w), T, slots, H, R, code,
         out.data_ptr(), dw.data_ptr())
    return out, dw


def route_grad(dslot_w, logits, ids, S=0, renormalize=True):
    """Gradient of `route_sort`'s routed weights: dlogits fp32 [T][E] from
    dslot_w fp32 [T*(k+S)], the logits and the picked ids [T][k]."""
    _need(logits.dim() == 2 and ids.dim() == 2, "logits must be [T][E] and ids [T][k]")
    dev = logits.device
    T, E = logits.shape
    k = ids.shape[1]
    if (T | E | k | S) >> 31:
        _too_large(T, E, k, S)
    _tensor("logits", logits, torch.float32, logits.shape)
    _tensor("ids", ids, torch.int32, (T, k), dev)
    _need(S >= 0 and dslot_w.numel() == T * (k + S), f"dslot_w must hold {T} x {k + S} entries")
    _tensor("dslot_w", dslot_w, torch.float32, dslot_w.shape, dev)
    out = torch.empty_like(logits)
    _run("milo_route_grad", dev, dslot_w.data_ptr(), logits.data_ptr(), ids.data_ptr(), T, E, k, S,
         1 if renormalize else 0, out.data_ptr())
    return out


# ------------------------------------------------------------------ products

def _weights(w):
    """(E, N, K) of a [N][K] or [E][N][K] weight tensor."""
    _need(w.dim() in (2, 3), "w must be [N][K] or [E][N][K]")
    if w.numel() >> 31 and max(w.shape) >> 31:
        _too_large(*w.shape)
    return (1, *w.shape) if w.dim() == 2 else tuple(w.shape)


def _offsets(offsets, E, dev):
    if offsets is not None:
        _tensor("offsets", offsets, torch.int32, (E + 1,), dev)
    else:
        _need(E == 1, f"offsets is required with {E} experts")


def _act(activation):
    _need(activation in _ACTS, f"unknown activation {activation!r}: one of {', '.join(_ACTS)}")
    return _ACTS[activation]


def moe_linear(x, w, offsets=None, bias=None, activation="none", mul=None, residual=None, out_dtype=None,
               return_pre=False, max_rows_per_expert=0, out=None):
    """Grouped product y = act(x w[e]^T + bias[e]) * mul + residual over the
    rows [offsets[e], offsets[e+1]) of each expert (see include/milo.h).

    x [rows][K] and w [N][K] or [E][N][K], fp16 or bf16; offsets int32 [E+1]
    (None: one expert owns every row); bias [E][N] ([N] for one expert); mul,
    residual [rows][N]; activation "none", "relu", "silu", "gelu" or
    "gelu_tanh".  Returns y [rows][N] in x's type or out_dtype float32, and
    with return_pre also the pre-activation in x's type.  Rows outside the
    offsets are not written (a new tensor is uninitialised there).  out: may be
    mul or residual itself where the types are equal, and shares no memory with
    another operand.
    max_rows_per_expert: a bound the caller knows, for the kernel choice.
    Scratch: with K no multiple of 8 (or w off a 16-byte address) and many rows
    it holds a copy of w in whole rows, made in every call."""
    code = _float_type("x", x, wide=False)
    _need(x.dim() == 2, "x must be [rows][K]")
    dev, dt = x.device, x.dtype
    E, N, K = _weights(w)
    R = x.shape[0]
    if R >> 31 or max_rows_per_expert > 0x7FFFFFFF:
        _too_large(R, max_rows_per_expert)
    _tensor("x", x, dt, (R, K))
    _tensor("w", w, dt, w.shape, dev)
    _offsets(offsets, E, dev)
    if bias is not None:
        _tensor("bias", bias, dt, (N,) if bias.dim() == 1 and E == 1 else (E, N), dev)
    if mul is not None:
        _tensor("mul", mul, dt, (R, N), dev)
    if residual is not None:
        _tensor("residual", residual, dt, (R, N), dev)
    odt = dt if out_dtype is None else out_dtype
    _need(odt in (dt, torch.float32), f"out_dtype must be {dt} or torch.float32")
    if out is None:
        out = torch.empty((R, N), dtype=odt, device=dev)
    else:
        _tensor("out", out, odt, (R, N), dev)
        _apart(out, x, w, offsets, bias, same=(mul, residual))
    pre = torch.empty((R, N), dtype=dt, device=dev) if return_pre else None
    ref = C.byref(L.MiloLinearDesc(
        E, N, K, R, max_rows_per_expert, code, L.F32 if odt is torch.float32 else code, _act(activation), x.data_ptr(),
        w.data_ptr(), _ptr(offsets), _ptr(bias), _ptr(mul), _ptr(residual), _ptr(pre), out.data_ptr()))
    nbytes = _call("milo_moe_linear_workspace_bytes", dev, ref)
    ws = _scratch(nbytes, dev)
    _run("milo_moe_linear", dev, ref, _ptr(ws), nbytes)
    return (out, pre) if return_pre else out


def moe_linear_act_grad(dy, pre, activation, mul=None, offsets=None, num_experts=None, bias_grad=False):
    """Gradient through `moe_linear`'s epilogue: (dpre, dmul, dbias) with
    dpre = dy * mul * act'(pre), dmul = dy * act(pre) (None without mul) and
    dbias fp32 [E][N], the sum of dpre over each expert's rows (None unless
    bias_grad).  The residual's gradient is dy itself.  Rows outside the
    offsets are not written (uninitialised)."""
    code = _float_type("dy", dy, wide=False)
    _need(dy.dim() == 2, "dy must be [rows][N]")
    dev, dt = dy.device, dy.dtype
    R, N = dy.shape
    E = num_experts if num_experts is not None else 1 if offsets is None else offsets.numel() - 1
    if (R | N) >> 31 or E > 0x7FFFFFFF:
        _too_large(R, N, E)
    _tensor("dy", dy, dt, (R, N))
    _tensor("pre", pre, dt, (R, N), dev)
    if mul is not None:
        _tensor("mul", mul, dt, (R, N), dev)
    _offsets(offsets, E, dev)
    dpre = torch.empty_like(dy)
    dmul = None if mul is None else torch.empty_like(dy)
    dbias = torch.empty((E, N), dtype=torch.float32, device=dev) if bias_grad else None
    nbytes = L.lib().milo_moe_linear_act_grad_workspace_bytes(E, N, R) if bias_grad else 0
    ws = _scratch(nbytes, dev)
    _run("milo_moe_linear_act_grad", dev, dy.data_ptr(), pre.data_ptr(), _ptr(mul), _ptr(offsets), E, N, R, code,
         _act(activation), dpre.data_ptr(), _ptr(dmul), _ptr(dbias), _ptr(ws), nbytes)
    return dpre, dmul, dbias


def moe_linear_grad(dy, x, w, offsets=None, need_dx=True, need_dw=True, dw_dtype=None, dx_add=None):
    """Gradients of the product: (dx [rows][K] = dy w[e], dw like w = sum over
    each expert's rows of dy^T x), None where not needed.  dw in x's type or
    dw_dtype float32.  dx_add [rows][K]: added to dx in fp32 before its
    rounding (the gradient of the same x from another product).  Rows of dx
    outside the offsets are not written (uninitialised)."""
    code = _float_type("dy", dy, wide=False)
    _need(dy.dim() == 2 and x.dim() == 2, "dy must be [rows][N] and x [rows][K]")
    dev, dt = dy.device, dy.dtype
    E, N, K = _weights(w)
    R = dy.shape[0]
    if R >> 31:
        _too_large(R)
    _tensor("dy", dy, dt, (R, N))
    _tensor("x", x, dt, (R, K), dev)
    _tensor("w", w, dt, w.shape, dev)
    _offsets(offsets, E, dev)
    odt = dt if dw_dtype is None else dw_dtype
    _need(odt in (dt, torch.float32), f"dw_dtype must be {dt} or torch.float32")
    dx = torch.empty((R, K), dtype=dt, device=dev) if need_dx else None
    dw = torch.empty(w.shape, dtype=odt, device=dev) if need_dw else None
    if dx_add is not None:
        _need(need_dx, "dx_add without dx")
        _tensor("dx_add", dx_add, dt, (R, K), dev)
    ref = C.byref(L.MiloLinearGradDesc(
        E, N, K, R, code, L.F32 if odt is torch.float32 else code, dy.data_ptr(), x.data_ptr(), w.data_ptr(),
        _ptr(offsets), _ptr(dx_add), _ptr(dx), _ptr(dw)))
    nbytes = _call("milo_moe_linear_grad_workspace_bytes", dev, ref)
    ws = _scratch(nbytes, dev)
    _run("milo_moe_linear_grad", dev, ref, _ptr(ws), nbytes)
    return dx, dw


class MoELayer16:
    """A routed SwiGLU MoE FFN with 16-bit experts, forward and backward: what
    `MoELayer` computes before its experts are quantized.  w1, w3 [E+S][F][H]
    (gate, up), w2 [E+S][H][F], fp16 or bf16."""

    def __init__(self, w1, w3, w2, E, k, S=0, renormalize=True):
        _need(w1.dim() == 3 and w1.shape == w3.shape and w1.shape[0] == E + S, "w1 and w3 must be [E+S][F][H]")
        _need(w2.shape == (E + S, w1.shape[2], w1.shape[1]), "w2 must be [E+S][H][F]")
        self.w1, self.w3, self.w2 = w1, w3, w2
        self.E, self.k, self.S, self.renormalize = E, k, S, renormalize

    def forward(self, x, logits, keep=False):
        """x [T][H] and float32 logits [T][E] to out [T][H]; with keep also what
        `backward` takes.  At most 65536 tokens (`route_sort`'s bound), or none."""
        T, slots = x.shape[0], self.k + self.S
        logits = logits.contiguous()
        _tensor("logits", logits, torch.float32, (T, self.E), self.w1.device)
        r = route_sort(logits, self.k, self.S, self.renormalize, own_scratch=True) if T else self._no_route(logits)
        off = r["offsets"]
        xs = moe_permute(x, r["pair_pos"], slots, dropped=False)
        up = moe_linear(xs, self.w3, off, max_rows_per_expert=T)
        got = moe_linear(xs, self.w1, off, activation="silu", mul=up, return_pre=keep, max_rows_per_expert=T)
        h, pre = got if keep else (got, None)
        y = moe_linear(h, self.w2, off, max_rows_per_expert=T)
        out = moe_unpermute(y, r["pair_pos"], slots, r["slot_w"])
        return (out, dict(route=r, logits=logits, xs=xs, up=up, pre=pre, h=h, y=y)) if keep else out

    def _no_route(self, logits):
        """What `route_sort` gives, for no token (it takes one at least)."""
        def of(dt, *shape):
            return torch.zeros(shape, dtype=dt, device=logits.device)
        i32, f32 = torch.int32, torch.float32
        return dict(ids=of(i32, 0, self.k), w=of(f32, 0, self.k), slot_w=of(f32, 0), sorted_pairs=of(i32, 0),
                    pair_pos=of(i32, 0), offsets=of(i32, self.E + self.S + 1))

    def backward(self, dout, kept, dw_dtype=None):
        """Gradients of x, the logits and the three weights for dout [T][H]."""
        r, slots = kept["route"], self.k + self.S
        off = r["offsets"]
        dy, dslot = moe_unpermute_grad(dout, kept["y"], r["pair_pos"], slots, r["slot_w"], dropped=False)
        dlogits = route_grad(dslot, kept["logits"], r["ids"], self.S, self.renormalize)
        dh, dw2 = moe_linear_grad(dy, kept["h"], self.w2, off, dw_dtype=dw_dtype)
        dpre, dup, _ = moe_linear_act_grad(dh, kept["pre"], "silu", mul=kept["up"], offsets=off)
        # xs feeds two products: the up product's half of its gradient is rounded to
        # 16 bits, the gate's is added to it in float32.  One more half step of the
        # type that the sum is rounded to next; a float32 half would be 4 bytes more
        # to write and to read for every value.
        dxs, dw3 = moe_linear_grad(dup, kept["xs"], self.w3, off, dw_dtype=dw_dtype)
        dxs, dw1 = moe_linear_grad(dpre, kept["xs"], self.w1, off, dw_dtype=dw_dtype, dx_add=dxs)
        return dict(dx=moe_permute_grad(dxs, r["pair_pos"], slots), dlogits=dlogits, dw1=dw1, dw3=dw3, dw2=dw2)
