"""Calls on tensors of a device that is not the current one (no GPU needed):
the binding runs against a stand-in for the library that records which device
was current and which stream was handed over."""
import types

import pytest
import torch

import extreme_quantized_moe_amd as m
from extreme_quantized_moe_amd import _lib


class Tensor:
    """A contiguous tensor on device 1, as far as the binding looks at it."""
    is_cuda = True

    def __init__(self, dtype, *shape):
        self.dtype, self.shape, self.device = dtype, torch.Size(shape), torch.device("cuda", 1)

    def is_contiguous(self):
        return True

    def contiguous(self):
        return self

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        return 4096


@pytest.fixture
def calls(monkeypatch):
    """The library's calls as (name, current device, arguments); device 0 is current outside them."""
    made, current = [], [0]

    class Device:
        def __init__(self, dev):
            self.index = torch.device(dev).index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *_):
            current[0] = self.before

    class Library:
        def __getattr__(self, name):
            def call(*args):
                made.append((name, current[0], args))
                return 512 if name.endswith("_bytes") else 0
            return call

    empty = torch.empty
    monkeypatch.setattr(_lib, "lib", lambda: Library())
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: Tensor(k["dtype"], *(
        a[0] if isinstance(a[0], (tuple, torch.Size)) else a)) if device is not None else empty(*a, **k))
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: types.SimpleNamespace(
        cuda_stream=700 + (current[0] if dev is None else torch.device(dev).index)))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 700 + i, raising=False)
    return made


def ran_on(calls, name):
    found = [(dev, args[-1]) for n, dev, args in calls if n == name]
    assert found, f"{name} was not called"
    return set(found)


def test_routing_runs_on_the_logits_device(calls):
    m.route_sort(Tensor(torch.float32, 6, 4), 2, own_scratch=True)
    assert ran_on(calls, "milo_route_sort") == {(1, 701)}


def test_workspaces_are_sized_for_the_tensors_device(calls):
    dt = torch.bfloat16
    x, w, dy = Tensor(dt, 40, 64), Tensor(dt, 32, 64), Tensor(dt, 40, 32)
    m.moe_linear(x, w)
    m.moe_linear_grad(dy, x, w)
    for name in ("milo_moe_linear", "milo_moe_linear_grad"):
        assert ran_on(calls, name) == {(1, 701)}
        assert {dev for dev, _ in ran_on(calls, name + "_workspace_bytes")} == {1}


def test_layer_runs_on_its_own_device(calls, monkeypatch):
    """Every call of a layer whose weights and inputs are on device 1."""
    dt = torch.float16
    monkeypatch.setattr(torch, "zeros", torch.empty)
    monkeypatch.setattr(torch, "empty_like", lambda t: Tensor(t.dtype, *t.shape))
    layer = m.MoELayer16(Tensor(dt, 4, 32, 64), Tensor(dt, 4, 32, 64), Tensor(dt, 4, 64, 32), 4, 2)
    _, kept = layer.forward(Tensor(dt, 6, 64), Tensor(torch.float32, 6, 4), keep=True)
    layer.backward(Tensor(dt, 6, 64), kept)
    on = {(n, dev) for n, dev, _ in calls if n not in ("milo_route_workspace_bytes",)}
    assert len(on) >= 10 and {dev for _, dev in on} == {1}, on
