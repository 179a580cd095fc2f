"""Sizes that the library's 32-bit numbers do not hold are refused by the torch
binding (no GPU needed): as ctypes passes them, 2^32 + 2 rows would be two."""
import pytest
import torch

import extreme_quantized_moe_amd as m

BIG = (1 << 32) + 2      # 2 where a 32-bit number is expected


@pytest.mark.parametrize("call", [
    lambda m, t, i, f: m.moe_permute(t(BIG, 1), i(4), 2),
    lambda m, t, i, f: m.moe_permute(t(2, BIG), i(4), 2),
    lambda m, t, i, f: m.moe_permute(t(2, 1), i(2 * BIG), BIG),
    lambda m, t, i, f: m.moe_unpermute(t(BIG, 1), i(4), 2),
    lambda m, t, i, f: m.moe_permute_grad(t(2, BIG), i(4), 2),
    lambda m, t, i, f: m.moe_unpermute_grad(t(2, 1), t(BIG, 1), i(4), 2),
    lambda m, t, i, f: m.moe_linear(t(BIG, 1), t(1, 1)),
    lambda m, t, i, f: m.moe_linear(t(2, BIG), t(1, BIG)),
    lambda m, t, i, f: m.moe_linear(t(2, 1), t(BIG, 1, 1), i(BIG + 1)),
    lambda m, t, i, f: m.moe_linear(t(2, 1), t(1, 1), max_rows_per_expert=BIG),
    lambda m, t, i, f: m.moe_linear_grad(t(BIG, 1), t(BIG, 1), t(1, 1)),
    lambda m, t, i, f: m.moe_linear_grad(t(2, BIG), t(2, 1), t(BIG, 1)),
    lambda m, t, i, f: m.moe_linear_act_grad(t(2, BIG), t(2, BIG), "silu"),
    lambda m, t, i, f: m.moe_linear_act_grad(t(2, 1), t(2, 1), "silu", num_experts=BIG),
    lambda m, t, i, f: m.route_grad(f(BIG), f(BIG, 1), i(BIG, 1)),
    lambda m, t, i, f: m.route_grad(f(BIG), f(2, 1), i(2, 1), S=BIG),
])
def test_binding_refuses_sizes_over_32_bits(call):
    def make(dt):
        return lambda *shape: torch.empty(shape, dtype=dt, device="meta")
    with pytest.raises(ValueError, match="32-bit"):
        call(m, make(torch.float16), make(torch.int32), make(torch.float32))


def test_binding_refuses_an_output_of_more_rows_than_32_bits(monkeypatch):
    from extreme_quantized_moe_amd import moe16
    monkeypatch.setattr(moe16, "_tensor", lambda *a: None)      # the operands' own checks aside
    with pytest.raises(ValueError, match="32-bit"):
        moe16.moe_permute(torch.empty((2, 1), dtype=torch.float16, device="meta"),
                          torch.empty(4, dtype=torch.int32, device="meta"), 2, num_rows=BIG)
