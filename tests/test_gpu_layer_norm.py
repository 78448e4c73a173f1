"""Layer norm on the GPU against 64 bits, forward and backward; tolerances are
derived beside the plain forms in rows_reference.py."""

import pytest
import torch

from rows_reference import (E4M3, INT8, U32, assert_near, moments64, norm64, norm_backward64, pack64)
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


def inputs(rows, cols, dtype, vector_dtype=FP32, seed=0):
    g = torch.Generator().manual_seed(seed + 31 * rows + cols)
    x = torch.empty(rows, cols).normal_(generator=g) * (0.5 + torch.empty(rows, 1).normal_(generator=g).abs()) + 0.3
    x[:, 3::97] *= 30  # a few columns far larger than the others
    dy = torch.empty(rows, cols).normal_(generator=g)
    weight = 1 + 0.2 * torch.empty(cols).normal_(generator=g)
    bias = 0.2 * torch.empty(cols).normal_(generator=g)
    return x.to(dtype), dy.to(dtype), weight.to(vector_dtype), bias.to(vector_dtype)


def check_forward(got, stats, x, weight, bias, center, eps=1e-5):
    want, room = norm64(x, weight, bias, eps, center)
    assert got.dtype == x.dtype
    assert_near(got, want, room)
    mean, rstd = moments64(x.reshape(-1, x.shape[-1]), eps, center)
    assert_near(stats[:, :1], mean, 48 * U32 * x.double().abs().reshape(-1, x.shape[-1]).mean(1, keepdim=True))
    assert_near(stats[:, 1:], rstd, 64 * U32 * rstd)


def check_backward(got, dy, x, weight, stats, center, bias):
    for g, (want, room) in zip(got, norm_backward64(dy, x, weight, stats.cpu(), center)):
        if g is not None:
            assert_near(g.reshape(want.shape), want, room)
    assert (got[1] is None) == (weight is None) and (got[2] is None) == (not bias)


# lanes of a warp, one to many rows a warp; CTAs of 2 to 32 warps; odd widths; rows that no CTA holds
CASES = [(1, 1), (3, 2), (2, 7), (5, 8), (70, 16), (9, 24), (1, 32), (257, 40), (100, 64), (33, 72), (130, 128), (7, 200),
         (64, 255), (64, 256), (65, 257), (20, 264), (3000, 264), (1, 2048), (301, 2048), (50, 1301), (19, 2056),
         (5, 4104), (3, 8192), (4, 8191), (2, 8193), (3, 8200), (9, 20000)]


@DTYPES
@pytest.mark.parametrize("center", [True, False], ids=["layer", "rms"])
@pytest.mark.parametrize("rows,cols", CASES)
def test_forward_and_backward(rows, cols, center, dtype):
    x, dy, weight, bias = inputs(rows, cols, dtype)
    dev = [t.cuda() for t in (x, weight, bias)]
    y, stats = ops.layer_norm(*dev, center=center)
    check_forward(y, stats, x, weight, bias, center)
    got = ops.layer_norm_backward(dy.cuda(), dev[0], dev[1], stats, center=center)
    check_backward(got, dy, x, weight, stats, center, True)
    again = ops.layer_norm_backward(dy.cuda(), dev[0], dev[1], stats, center=center)
    for a, b in zip(got, again):
        assert torch.equal(a, b), "the same call gives the same bits"


@FORMS
@DTYPES
@pytest.mark.parametrize("rows,cols", CASES)
def test_kept_in_8_bits(rows, cols, dtype, form):
    x, dy, weight, bias = inputs(rows, cols, dtype, seed=1)
    if rows * cols > 50000:
        x, dy = x[:6], dy[:6]
    center = rows % 2 == 0
    dev = [t.cuda() for t in (x, weight, bias)]
    y, stats, packed = ops.layer_norm(*dev, center=center, pack=form)
    plain = ops.layer_norm(*dev, center=center)
    assert torch.equal(y, plain[0]) and torch.equal(stats, plain[1])
    codes, exponents, values = pack64(x, form)
    assert torch.equal(packed.codes.float().cpu().double(), codes)
    assert torch.equal(packed.scales.cpu().long(), exponents + 127)
    got = ops.layer_norm_backward(dy.cuda(), packed, dev[1], stats, center=center)
    check_backward(got, dy, values, weight, stats, center, True)
    alone = ops.pack_activations(dev[0], form)
    assert torch.equal(alone.codes.view(torch.uint8), packed.codes.view(torch.uint8))
    assert torch.equal(alone.scales, packed.scales)


@pytest.mark.parametrize("vector_dtype", [FP32, BF16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("cols", [64, 77, 520])
def test_without_weight_or_bias(cols, vector_dtype):
    x, dy, weight, bias = inputs(12, cols, BF16, vector_dtype, seed=2)
    for w in (None, weight):
        for b in (None, bias):
            dev = [None if t is None else t.cuda() for t in (x, w, b)]
            y, stats = ops.layer_norm(*dev)
            check_forward(y, stats, x, w, b, True)
            got = ops.layer_norm_backward(dy.cuda(), dev[0], dev[1], stats, bias=b is not None)
            check_backward(got, dy, x, w, stats, True, b is not None)


def test_far_mean_and_sizes():
    # a mean a thousand times the deviation, tiny and large rows
    x, dy, weight, bias = inputs(8, 1024, FP32, seed=3)
    x[0] = x[0] * 1e-3 + 1.0
    x[1] *= 1e15
    x[2] *= 1e-15
    x[3] = 0
    x[4] = 7.0
    y, stats = ops.layer_norm(x.cuda(), weight.cuda(), bias.cuda())
    check_forward(y, stats, x, weight, bias, True)
    got = ops.layer_norm_backward(dy.cuda(), x.cuda(), weight.cuda(), stats)
    check_backward(got, dy, x, weight, stats, True, True)


@pytest.mark.parametrize("cols", [64, 100, 1000, 2048, 9000])
def test_a_row_that_is_not_finite_stays_alone(cols):
    x, dy, weight, bias = inputs(6, cols, FP32, seed=4)
    x[1, 5], x[3, 0], x[4, cols - 1] = float("inf"), float("nan"), float("-inf")
    y, stats, packed = ops.layer_norm(x.cuda(), weight.cuda(), bias.cuda(), pack=E4M3)
    keep = [0, 2, 5]
    check_forward(y[keep], stats[keep], x[keep], weight, bias, True)
    assert y[[1, 3, 4]].isnan().any(1).all()
    for kept in (x.cuda(), packed):
        dx, dw, db = ops.layer_norm_backward(dy.cuda(), kept, weight.cuda(), stats)
        values = x if kept is not packed else ops.unpack_activations(packed).cpu()
        assert_near(dx[keep], *[t[keep] for t in norm_backward64(dy, values, weight, stats.cpu(), True)[0]])
        assert dx[[1, 3, 4]].isnan().all() and dw.isnan().any()
        assert db.isfinite().all()


@DTYPES
@pytest.mark.parametrize("cols", [48, 130, 1024, 1031, 8200])
def test_strides_and_in_place(cols, dtype):
    x, dy, weight, bias = inputs(37, cols, dtype, seed=5)
    w, b = weight.cuda(), bias.cuda()
    wants = {}
    for lead, tail in ((0, 0), (8, 8), (1, 0), (3, 4), (8, 1)):
        buffer = torch.full((37, lead + cols + tail), float("nan"), dtype=dtype, device="cuda")
        view = buffer[:, lead:lead + cols]
        view.copy_(x)
        # one order of the sums for aligned rows, another for the others
        aligned = cols % 8 == 0 and lead % 8 == 0 and (lead + tail) % 8 == 0
        want = wants.setdefault(aligned, ops.layer_norm(view, w, b))
        check_forward(want[0], want[1], x, weight, bias, True)
        y, stats = ops.layer_norm(view, w, b)
        assert torch.equal(y, want[0]) or not aligned
        check_forward(y, stats, x, weight, bias, True)
        g = buffer.clone()[:, lead:lead + cols]
        g.copy_(dy)
        back = ops.layer_norm_backward(g, view, w, stats)
        check_backward(back, dy, x, weight, stats, True, True)
        for over in (g.clone(), g):  # onto dy, and onto x
            source = view if over is g else view.clone()
            got = ops.layer_norm_backward(g if over is g else over, source, w, stats, out=source if over is g else over)
            check_backward(got, dy, x, weight, stats, True, True)
        view.copy_(x)
        out, _ = ops.layer_norm(view, w, b, out=view)
        assert out.data_ptr() == view.data_ptr()
        check_forward(out, stats, x, weight, bias, True)
        assert buffer[:, :lead].isnan().all() and buffer[:, lead + cols:].isnan().all()


def test_leading_dimensions():
    x, dy, weight, bias = inputs(60, 96, BF16, seed=6)
    w, b = weight.cuda(), bias.cuda()
    want, stats = ops.layer_norm(x.cuda(), w, b)
    back = ops.layer_norm_backward(dy.cuda(), x.cuda(), w, stats)
    cube, dcube = x.cuda().view(3, 4, 5, 96), dy.cuda().view(3, 4, 5, 96)
    y, s = ops.layer_norm(cube, w, b)
    assert y.shape == cube.shape and torch.equal(y.view(60, 96), want) and torch.equal(s, stats)
    turned = cube.transpose(0, 1)  # no single row stride: copied
    y, s = ops.layer_norm(turned, w, b)
    assert torch.equal(y, want.view(3, 4, 5, 96).transpose(0, 1))
    got = ops.layer_norm_backward(dcube.transpose(0, 1), turned, w, s)
    assert torch.equal(got[0], back[0].view(3, 4, 5, 96).transpose(0, 1))
    row = ops.layer_norm(x[0].cuda(), w, b)
    assert torch.equal(row[0], want[0]) and row[1].shape == (1, 2)
    with pytest.raises(ValueError):
        ops.layer_norm(turned, w, b, out=turned)


def test_no_rows():
    w, b = torch.ones(40, device="cuda"), torch.ones(40, device="cuda")
    for shape in ((0, 40), (2, 0, 40)):
        x = torch.empty(shape, device="cuda")
        y, stats, packed = ops.layer_norm(x, w, b, pack=INT8)
        assert y.shape == shape and stats.shape == (0, 2)
        for kept in (x, packed):
            dx, dw, db = ops.layer_norm_backward(x, kept, w, stats)
            assert dx.shape == shape and (dw == 0).all() and (db == 0).all()
        assert ops.unpack_activations(packed).shape == shape


@pytest.mark.parametrize("vector_dtype", [FP32, BF16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("cols", [64, 520, 8200])
def test_vectors_and_their_gradients_in_flat_buffers(cols, vector_dtype):
    # weight and bias read from, and gradients written to, odd offsets of flat buffers
    x, dy, weight, bias = inputs(45, cols, BF16, vector_dtype, seed=7)
    flat = torch.full((2 * cols + 20,), 7.0, dtype=vector_dtype, device="cuda")
    grad = flat.clone()
    spots = slice(3, 3 + cols), slice(9 + cols, 9 + 2 * cols)
    flat[spots[0]] = weight.cuda()
    flat[spots[1]] = bias.cuda()
    y, stats = ops.layer_norm(x.cuda(), flat[spots[0]], flat[spots[1]])
    check_forward(y, stats, x, weight, bias, True)
    want = ops.layer_norm_backward(dy.cuda(), x.cuda(), weight.cuda(), stats)
    got = ops.layer_norm_backward(dy.cuda(), x.cuda(), flat[spots[0]], stats, weight_out=grad[spots[0]],
                                  bias_out=grad[spots[1]])
    assert torch.equal(got[0], want[0])
    for i, s in enumerate(spots):
        assert torch.equal(grad[s], want[1 + i].to(vector_dtype))
        grad[s] = 7.0
    assert (grad == 7.0).all()


def test_gradients_against_differences():
    x, dy, weight, bias = [t.double() for t in inputs(20, 96, FP32, seed=8)]
    g = torch.Generator().manual_seed(9)
    args = [t.float().cuda() for t in (x, weight, bias)]
    y, stats = ops.layer_norm(*args)
    grads = ops.layer_norm_backward(dy.float().cuda(), args[0], args[1], stats)
    for i in range(3):
        direction = torch.empty(args[i].shape).normal_(generator=g).cuda()
        step, value = 1e-2, []
        for sign in (1, -1):
            moved = list(args)
            moved[i] = args[i] + sign * step * direction
            value.append(float((ops.layer_norm(*moved)[0].double() * dy.cuda()).sum()))
        slope = (value[0] - value[1]) / (2 * step)
        want = float((grads[i].double() * direction).sum())
        # third-order term of a central difference (step^2) and fp32 outputs, both against the gradient's size
        assert abs(slope - want) <= 2e-3 * float(grads[i].double().norm()), i


def test_streams_and_capture():
    x, dy, weight, bias = [t.cuda() for t in inputs(900, 1024, BF16, seed=10)]
    y, stats, packed = ops.layer_norm(x, weight, bias, pack=E4M3)
    want = ops.layer_norm_backward(dy, packed, weight, stats)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = ops.layer_norm_backward(dy, packed, weight, stats)
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(want, other):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    static = torch.zeros_like(x)
    with torch.cuda.graph(graph):
        gy, gstats, gpacked = ops.layer_norm(static, weight, bias, pack=E4M3)
        got = ops.layer_norm_backward(dy, gpacked, weight, gstats)
    for _ in range(2):
        static.copy_(x)
        graph.replay()
        assert torch.equal(gy, y)
        for a, b in zip(want, got):
            assert torch.equal(a, b)


def test_offsets_past_32_bits():
    rows, cols = 40, 64
    stride = (1 << 31) // (rows - 2) // 64 * 64 + 64
    big = torch.empty((rows - 1) * stride + cols, dtype=BF16, device="cuda")
    x, dy, weight, bias = [t.cuda() for t in inputs(rows, cols, BF16, seed=11)]
    view = big.as_strided((rows, cols), (stride, 1))
    want, stats, packed = ops.layer_norm(x, weight, bias, pack=INT8)
    back = ops.layer_norm_backward(dy, x, weight, stats)
    view.copy_(x)
    got, _, kept = ops.layer_norm(view, weight, bias, pack=INT8, out=view)
    assert torch.equal(got, want) and torch.equal(kept.codes, packed.codes)
    ops.unpack_activations(packed, out=view)
    assert torch.equal(view, ops.unpack_activations(packed))
    view.copy_(dy)
    got = ops.layer_norm_backward(view, x, weight, stats, out=view)
    for a, b in zip(got, back):
        assert torch.equal(a, b)


def leaves(rows=30, cols=72, dtype=FP32, vector_dtype=FP32):
    x, dy, weight, bias = inputs(rows, cols, dtype, vector_dtype, seed=12)
    return [t.cuda().requires_grad_() for t in (x, weight, bias)], dy.cuda()


@pytest.mark.parametrize("pack", [None, E4M3, INT8], ids=["whole", "e4m3", "int8"])
def test_autograd(pack):
    args, dy = leaves()
    y = ops.layer_norm_autograd(*args, pack=pack)
    y.backward(dy)
    plain = [t.detach() for t in args]
    want, stats, *packed = ops.layer_norm(*plain, pack=pack)
    grads = ops.layer_norm_backward(dy, packed[0] if packed else plain[0], plain[1], stats)
    assert torch.equal(y, want)
    for a, g in zip(args, grads):
        assert torch.equal(a.grad, g)


def test_autograd_of_broadcast_and_strided_gradients():
    args, _ = leaves(vector_dtype=BF16)
    ops.layer_norm_autograd(*args).sum().backward()  # a gradient with strides of zero
    got = [a.grad.clone() for a in args]
    for a in args:
        a.grad = None
    ops.layer_norm_autograd(*args).backward(torch.ones(30, 72, device="cuda"))
    for a, g in zip(args, got):
        assert torch.equal(a.grad, g) and a.grad.dtype == a.dtype
    # an input whose columns are not contiguous, an input without a gradient
    x = args[0].detach().t().contiguous().t().requires_grad_()
    y = ops.layer_norm_autograd(x, args[1].detach(), None)
    y.sum().backward()
    want = ops.layer_norm_autograd(args[0].detach().clone().requires_grad_(), args[1].detach(), None)
    assert torch.equal(y, want) and x.grad is not None


def test_second_derivatives_are_refused():
    args, _ = leaves()
    grads = torch.autograd.grad(ops.layer_norm_autograd(*args).square().sum(), args, create_graph=True)
    with pytest.raises(RuntimeError):
        (sum(g.square().sum() for g in grads) + args[0].square().sum()).backward()


def test_inputs_that_require_gradients():
    args, dy = leaves()
    plain = [t.detach() for t in args]
    _, stats = ops.layer_norm(*plain)
    for i in range(3):
        some = list(plain)
        some[i] = args[i]
        with pytest.raises(ValueError):
            ops.layer_norm(*some)
    with pytest.raises(ValueError):
        ops.layer_norm_backward(dy, args[0], plain[1], stats)
    with pytest.raises(ValueError):
        ops.layer_norm_backward(dy.requires_grad_(), plain[0], plain[1], stats)
    with torch.no_grad():
        assert torch.equal(ops.layer_norm(*args)[0], ops.layer_norm(*plain)[0])


def test_tensor_checks():
    x, dy, weight, bias = [t.cuda() for t in inputs(6, 64, FP32, seed=13)]
    _, stats, packed = ops.layer_norm(x, weight, bias, pack=E4M3)
    for bad in (x.half(), x.t(), x.cpu(), x[:, :0], torch.tensor(1.0, device="cuda")):
        with pytest.raises(ValueError):
            ops.layer_norm(bad, weight, bias)
    for w, b in ((weight[:5], bias), (weight.bfloat16(), bias), (weight, bias.cpu()), (weight.double(), bias.double()),
                 (weight.expand(2, 64)[0:1], bias)):
        with pytest.raises(ValueError):
            ops.layer_norm(x, w, b)
    for out in (x[:5], x.bfloat16(), x.t().contiguous().t(), x[:1].expand(6, 64)):
        with pytest.raises(ValueError):
            ops.layer_norm(x, weight, bias, out=out)
    with pytest.raises(ValueError):
        ops.layer_norm(x, weight, bias, pack=torch.float8_e5m2)
    with pytest.raises(ValueError):
        ops.layer_norm(x[:-1], weight, bias, out=x[1:])
    for g, s, st in ((dy[:5], x, stats), (dy.bfloat16(), x, stats), (dy, x, stats[:5]), (dy, x, stats.double()),
                     (dy[:5], packed, stats[:5]), (dy[:, :32], packed, stats), (dy.view(2, 3, 64), packed, stats)):
        with pytest.raises(ValueError):
            ops.layer_norm_backward(g, s, weight, st)
    vector = torch.empty(100, device="cuda")
    for more in (dict(out=x[:5]), dict(weight_out=vector[:63]), dict(weight_out=vector[:64], bias_out=vector[30:94]),
                 dict(weight_out=vector[:64].bfloat16(), bias_out=vector[:64]), dict(bias=False, bias_out=vector[:64]),
                 dict(weight_out=x[2]), dict(bias_out=dy[0])):
        with pytest.raises(ValueError):
            ops.layer_norm_backward(dy, x, weight, stats, **more)
