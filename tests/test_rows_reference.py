"""The 64-bit forms for large matrices equal the ones written group by group and
token by token (not gpu)."""

import pytest
import torch

from rows_reference import E4M3, INT8, embedding_backward64, embedding_backward64_many, pack64, pack64_many


@pytest.mark.parametrize("form", [E4M3, INT8], ids=["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("cols", [64, 71])
def test_pack(cols, dtype, form):
    limit = 448.0 if form == E4M3 else 127.0
    g = torch.Generator().manual_seed(cols)
    x = torch.empty(60, cols).normal_(generator=g) * torch.empty(60, cols).normal_(0, 4, generator=g).exp()
    above = torch.nextafter(torch.tensor(limit), torch.tensor(1e9))
    for r, top in enumerate((limit, above, limit / 2, 2 * above, -limit, 2.0 ** -140, 2.0 ** -126 * limit, 3.3e38, 0.0)):
        x[r] = x[r].clamp(-1, 1) * abs(float(top)) / 4
        x[r, 3] = float(top)
    x[10, 2], x[11, cols - 1], x[12, 40] = float("nan"), float("inf"), float("-inf")
    x[13] = torch.linspace(-limit, limit, cols)
    x[14, :32] = torch.arange(32) / 16 * limit / 2
    x = x.to(dtype)
    for got, want in zip(pack64_many(x, form), pack64(x, form)):
        assert got.dtype == want.dtype and torch.equal(got.nan_to_num(0.5), want.nan_to_num(0.5))
        assert torch.equal(got.isnan(), want.isnan())


def test_embedding_gradient():
    g = torch.Generator().manual_seed(1)
    ids = torch.randint(-2, 13, (300,), generator=g)
    dy = torch.empty(300, 7).normal_(generator=g)
    for got, want in zip(embedding_backward64_many(dy, ids, 11, 2.5), embedding_backward64(dy, ids, 11, 2.5)):
        assert torch.allclose(got, want, rtol=1e-13, atol=1e-13)
