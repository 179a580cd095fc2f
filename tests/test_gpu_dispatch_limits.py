"""Rows to the experts and back at the most tokens a call takes."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_most_tokens_with_rows_of_many_pieces():
    """2^24 rows of 131 values: 256 threads a token are 2^32, more than one launch takes."""
    import extreme_quantized_moe_amd as m
    T, H = 1 << 24, 131
    x = torch.randint(-9, 9, (T, H), dtype=torch.int8, device="cuda").to(torch.float16)
    x[:, 0] = torch.arange(T, device="cuda").remainder(2039).to(torch.float16)
    pos = torch.arange(T - 1, -1, -1, dtype=torch.int32, device="cuda")
    y = m.moe_permute(x, pos, 1)
    assert all(torch.equal(y[T - a - 4096:T - a].flip(0), x[a:a + 4096]) for a in range(0, T, 4096))
    w = torch.full((T,), 2.0, device="cuda")
    w[5] = w[T - 5] = 0.5
    out = m.moe_unpermute(y, pos, 1, w)
    del y
    # the values are whole numbers under 2048: doubled and halved exactly
    assert torch.equal(out, x * w[:, None].to(torch.float16))
