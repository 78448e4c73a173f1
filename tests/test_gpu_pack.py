"""Activations in 8 bits on the GPU: codes, scales and values equal the 64-bit
definition bit for bit."""

import pytest
import torch

from rows_reference import E4M3, INT8, pack64
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


def inputs(rows, cols, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + 7 * rows + cols)
    x = torch.empty(rows, cols).normal_(generator=g)
    return (x * torch.empty(rows, cols).normal_(0, 3, generator=g).exp()).to(dtype)


def check(x, form, packed):
    codes, exponents, values = pack64(x, form)
    assert packed.codes.dtype == packed.form == form and packed.shape == x.shape and packed.dtype == x.dtype
    assert torch.equal(packed.codes.float().cpu().double(), codes)
    assert torch.equal(packed.scales.cpu().long(), exponents + 127)
    for dtype in (None, FP32, BF16):
        got = ops.unpack_activations(packed, dtype)
        want = values.to(dtype or x.dtype)
        assert got.dtype == want.dtype
        assert torch.equal(got.cpu().nan_to_num(12345.0), want.nan_to_num(12345.0))


@FORMS
@DTYPES
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 2), (5, 8), (2, 31), (7, 32), (9, 33), (11, 40), (300, 16), (4, 100),
                                       (3, 256), (2, 1000), (3, 777), (1, 2048), (2, 2049), (1, 8200), (2, 5000)])
def test_pack_and_unpack(rows, cols, dtype, form):
    x = inputs(rows, cols, dtype)
    check(x, form, ops.pack_activations(x.cuda(), form))


@FORMS
@DTYPES
@pytest.mark.parametrize("cols", [64, 65])
def test_borders(cols, dtype, form):
    """Largest entries around a power's limit, ties, signed zeros, subnormals, the type's ends."""
    limit = 448.0 if form == E4M3 else 127.0
    x = torch.zeros(40, cols)
    for r in range(16):
        x[r, 0] = limit * 2.0 ** (r - 8)
        x[r, 1:33] = torch.arange(32) / 16 * 2.0 ** (r - 8)  # ties of either form among them
    above = torch.nextafter(torch.tensor(limit), torch.tensor(1e9))
    x[16, 0], x[17, 0], x[18, 0] = above, -above, limit
    x[16:19, 1] = 0.5
    x[19, 0], x[19, 1] = torch.finfo(dtype).max, 1.0
    x[20, 0], x[20, 1] = torch.finfo(dtype).smallest_normal, -torch.finfo(dtype).smallest_normal / 2
    x[21] = torch.finfo(dtype).smallest_normal / 4
    x[22] = -0.0
    x[23, :4] = torch.tensor([1.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -11])
    x[24, 40] = float("nan")
    x[25, 3] = float("inf")
    x[26, cols - 1] = float("-inf")
    x[27] = torch.linspace(-limit, limit, cols)
    x[28:] = inputs(12, cols, FP32)
    x = x.to(dtype)
    check(x, form, ops.pack_activations(x.cuda(), form))


@FORMS
@pytest.mark.parametrize("lead,tail", [(0, 0), (8, 8), (1, 0), (4, 4), (3, 2)])
def test_strides(lead, tail, form):
    x = inputs(21, 200, BF16, seed=3)
    buffer = torch.full((21, lead + 200 + tail), 5.0, dtype=BF16, device="cuda")
    view = buffer[:, lead:lead + 200]
    view.copy_(x)
    packed = ops.pack_activations(view, form)
    check(x, form, packed)
    values = ops.unpack_activations(packed)
    got = ops.unpack_activations(packed, out=view)
    assert got is view and torch.equal(view, values)
    assert (buffer[:, :lead] == 5.0).all() and (buffer[:, lead + 200:] == 5.0).all()


def test_shapes_and_reuse():
    x = inputs(24, 48, FP32, seed=4).cuda()
    packed = ops.pack_activations(x.view(2, 3, 4, 48), INT8)
    assert ops.unpack_activations(packed).shape == (2, 3, 4, 48)
    want = ops.pack_activations(x, INT8)
    assert torch.equal(packed.codes, want.codes)
    turned = x.view(4, 6, 48).transpose(0, 1)
    assert torch.equal(ops.unpack_activations(ops.pack_activations(turned, INT8)),
                       ops.unpack_activations(want).view(4, 6, 48).transpose(0, 1))
    row = ops.pack_activations(x[0], INT8)
    assert ops.unpack_activations(row).shape == (48,)
    codes = packed.data.data_ptr()
    again = ops.pack_activations((2 * x).view(2, 3, 4, 48), INT8, out=packed)
    assert again.data.data_ptr() == codes
    assert torch.equal(ops.unpack_activations(again).view(24, 48), 2 * ops.unpack_activations(want))
    needs = x.clone().requires_grad_()
    assert not ops.unpack_activations(ops.pack_activations(needs, INT8)).requires_grad


def test_no_rows():
    for shape in ((0, 40), (3, 0, 40)):
        packed = ops.pack_activations(torch.empty(shape, device="cuda"))
        assert ops.unpack_activations(packed).shape == shape


def test_capture():
    x = inputs(100, 300, BF16, seed=5).cuda()
    want = ops.unpack_activations(ops.pack_activations(x))
    static, graph = torch.zeros_like(x), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ops.unpack_activations(ops.pack_activations(static))
    static.copy_(x)
    graph.replay()
    assert torch.equal(got, want)


def test_tensor_checks():
    x = inputs(6, 64, FP32, seed=6).cuda()
    packed = ops.pack_activations(x)
    for bad in (x.half(), x.t(), x.cpu(), x[:, :0]):
        with pytest.raises(ValueError):
            ops.pack_activations(bad)
    for bad in (torch.float8_e5m2, torch.uint8, torch.bfloat16):
        with pytest.raises(ValueError):
            ops.pack_activations(x, bad)
    for bad in (x[:5], x.bfloat16(), x.view(2, 3, 64)):
        with pytest.raises(ValueError):
            ops.pack_activations(bad, out=packed)
    with pytest.raises(ValueError):
        ops.pack_activations(x, INT8, out=packed)
    buffer = torch.zeros(2048, dtype=torch.uint8, device="cuda")
    inside, beside = (buffer[at:at + 1536].view(FP32).view(6, 64) for at in (256, 400))
    over = ops.PackedActivations(buffer[:396], E4M3, (6, 64), FP32)
    with pytest.raises(ValueError):
        ops.pack_activations(inside, out=over)
    ops.pack_activations(beside, out=over)
    good = (packed.data, E4M3, (6, 64), FP32)
    assert torch.equal(ops.unpack_activations(ops.PackedActivations(*good)), ops.unpack_activations(packed))
    for i, bad in ((0, packed.data[:-1]), (0, packed.data.cpu()), (0, packed.data.view(torch.int8)),
                   (0, packed.data.view(6, 66)), (0, packed.data.expand(2, 396)[:, ::2].reshape(-1)[:395]),
                   (1, torch.uint8), (2, (6, 65)), (2, (6, 0)), (2, ()), (2, (-6, 64)), (2, (5, 64)), (3, torch.half)):
        args = list(good)
        args[i] = bad
        with pytest.raises(ValueError):
            ops.PackedActivations(*args)
    with pytest.raises(ValueError):
        ops.unpack_activations(packed, torch.half)
    for out in (x[:5], x.half(), x.t().contiguous().t()):
        with pytest.raises(ValueError):
            ops.unpack_activations(packed, out=out)
    with pytest.raises(ValueError):
        ops.unpack_activations(packed, BF16, out=x)
    with pytest.raises(ValueError):
        ops.unpack_activations(over, out=inside)
