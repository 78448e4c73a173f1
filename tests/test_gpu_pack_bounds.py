"""How far an entry of the 8-bit form may be off, as documented: e4m3 by 2^-4 of
itself or 2^-10 of the scale, whole numbers by half a scale, 1 / 127 of the
group's largest; what rounds up to 2^128 reads as inf."""

import pytest
import torch

from rows_reference import E4M3, GROUP, INT8, power_of_two
from zero_sharded_mixed_flatparameter_gb300 import binding as B
from zero_sharded_mixed_flatparameter_gb300 import ops

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32
DTYPES = pytest.mark.parametrize("dtype", [FP32, BF16], ids=["fp32", "bf16"])
FORMS = pytest.mark.parametrize("form", [E4M3, INT8], ids=["e4m3", "int8"])


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_sharded_mixed_flatparameter_gb300 import build_lib
    build_lib.build()
    B.load()


@FORMS
@DTYPES
def test_bounds(dtype, form):
    g = torch.Generator().manual_seed(3)
    x = torch.empty(4000, GROUP).normal_(generator=g) * torch.empty(4000, GROUP).normal_(0, 4, generator=g).exp()
    x[1000:2000] = torch.empty(1000, GROUP).uniform_(-1, 1, generator=g)
    x[2000:3000, 0] = torch.linspace(63.5, 127, 1000)  # whole numbers' scale near its largest share of the entry
    x[2000:3000, 1:] = torch.empty(1000, GROUP - 1).uniform_(-40, 40, generator=g).round() + 0.5
    x[3000, :2] = torch.tensor([63.75, 0.5])           # rounds to 0: off by more than 2^-7 of 63.75
    x[3001, :2] = torch.tensor([448.0, 2.0 ** -11])    # becomes 0: off by itself
    x[3002:3100] *= 2.0 ** -110
    x = x.to(dtype)
    packed = ops.pack_activations(x.cuda(), form)
    off = (ops.unpack_activations(packed, FP32).cpu().double() - x.double()).abs()
    scale = power_of_two(packed.scales.cpu().long() - 127)
    top = x.double().abs().amax(1, keepdim=True)
    if form == E4M3:
        assert (off <= torch.maximum(2.0 ** -4 * x.double().abs(), 2.0 ** -10 * scale)).all()
        assert (top > 224 * scale).all()
        assert off[3001, 1] == 2.0 ** -11
    else:
        assert (off <= scale / 2).all() and (off <= top / 127).all()
        assert off[3000, 1] == 0.5 > 63.75 / 128


@FORMS
@DTYPES
def test_the_ends_of_the_range(dtype, form):
    # the smallest magnitude that reads as inf, and its neighbour below
    border = 31 / 32 if form == E4M3 else 127 / 128
    bits = torch.int32 if dtype == FP32 else torch.int16
    at = torch.tensor(border * 2.0 ** 127).double().mul(2).to(dtype)
    assert float(at) == border * 2.0 ** 128
    if form == INT8:
        at = (at.view(bits) + 1).view(dtype)  # at the border itself the smaller scale still holds 127
    below = (at.view(bits) - 1).view(dtype)
    x = torch.zeros(4, GROUP, dtype=dtype)
    x[0, 3], x[1, 3], x[2, 3], x[3, 3] = at, below, -torch.finfo(dtype).max, -below
    x[:, 4] = 2.0 ** 100
    for out in (FP32, BF16):
        got = ops.unpack_activations(ops.pack_activations(x.cuda(), form), out).cpu()
        assert got[0, 3] == float("inf") and got[2, 3] == float("-inf")
        assert got[[1, 3]].isfinite().all() and not got.isnan().any()
        assert abs(float(got[1, 3]) - float(below)) <= float(below) / (16 if form == E4M3 else 127)
