"""Embedding lookup and its gradient on the GPU against 64 bits; tolerances are
derived beside the plain forms in rows_reference.py."""

import pytest
import torch

from rows_reference import U32, assert_near, embedding_backward64
from zero_sharded_mixed_flatparameter_gb300 import binding as B
from zero_sharded_mixed_flatparameter_gb300 import ops

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32
DTYPES = pytest.mark.parametrize("dtype", [FP32, BF16], ids=["fp32", "bf16"])


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_sharded_mixed_flatparameter_gb300 import build_lib
    build_lib.build()
    B.load()


def make_ids(tokens, rows, kind, seed=0, dtype=torch.int64):
    g = torch.Generator().manual_seed(seed + tokens + rows)
    if kind == "text":  # the probability falls as 1 / id
        ids = (torch.rand(tokens, generator=g, dtype=torch.float64) * torch.log(torch.tensor(rows + 1.0))).exp().long() - 1
        ids.clamp_(0, rows - 1)
    elif kind == "one":
        ids = torch.full((tokens,), rows // 2)
    else:
        ids = torch.randint(0, rows, (tokens,), generator=g)
    if tokens > 3 and kind != "one":  # padding, and what is no row
        ids[tokens // 3], ids[tokens - 1], ids[0] = -1, rows, -rows - 5
        if dtype == torch.int64:
            ids[1] = (1 << 32) + 1
    return ids.to(dtype)


def normal(*shape, dtype=FP32, seed=0):
    g = torch.Generator().manual_seed(seed + sum(shape))
    return torch.empty(shape).normal_(generator=g).to(dtype)


def looked_up(ids, table, scale):
    live = (ids >= 0) & (ids < table.shape[0])
    if table.shape[0] == 0:
        return torch.zeros(*ids.shape, table.shape[1], dtype=torch.float64)
    return scale * table.double()[torch.where(live, ids, 0).long()] * live[..., None]


CASES = [  # tokens, rows, dim, how ids are spread
    (1, 1, 1, "text"), (1, 100, 64, "any"), (2, 3, 8, "any"), (5, 2, 7, "text"), (31, 9, 33, "text"), (32, 40, 16, "one"),
    (33, 40, 16, "one"), (64, 5, 40, "one"), (65, 1000, 24, "any"), (700, 50, 264, "text"), (1000, 1, 100, "one"),
    (1500, 700, 321, "text"), (2000, 3, 12, "text"), (3001, 3000, 64, "any"), (1025, 153, 8, "text"),
    (100, 5000, 2056, "any"), (4000, 5, 2048, "text"), (90, 20, 4100, "text"), (2500, 60000, 16, "text"),
    (400, 260000, 8, "any"), (20000, 3, 8, "one"), (9000, 2, 24, "text"), (17000, 200, 16, "text"),
    (1300, 90, 511, "text"), (1300, 90, 513, "text"), (700, 300, 1001, "any"), (600, 4, 777, "one")]


@pytest.mark.parametrize("id_dtype", [torch.int32, torch.int64], ids=["int32", "int64"])
@DTYPES
@pytest.mark.parametrize("tokens,rows,dim,kind", CASES)
def test_lookup_and_gradient(tokens, rows, dim, kind, dtype, id_dtype):
    ids, scale = make_ids(tokens, rows, kind, dtype=id_dtype), 1.0 if tokens % 2 else 3.7
    table, dy = normal(rows, dim, dtype=dtype), normal(tokens, dim, dtype=dtype, seed=1)
    factor = float(torch.tensor(scale, dtype=FP32))
    got = ops.embedding(ids.cuda(), table.cuda(), scale=scale)
    want = looked_up(ids, table, factor)
    assert got.dtype == dtype
    assert_near(got, want, 2 * U32 * want.abs() if scale != 1.0 else 0.0)
    grad = ops.embedding_backward(dy.cuda(), ids.cuda(), rows, scale=scale)
    want, room = embedding_backward64(dy, ids, rows, factor)
    assert grad.dtype == dtype
    assert_near(grad, want, room)
    other = FP32 if dtype == BF16 else BF16
    out = torch.full((rows, dim), float("nan"), dtype=other, device="cuda")
    assert ops.embedding_backward(dy.cuda(), ids.cuda(), rows, scale=scale, out=out) is out
    assert_near(out, want, room)
    again = torch.full((rows, dim), float("nan"), dtype=other, device="cuda")
    ops.embedding_backward(dy.cuda(), ids.cuda(), rows, scale=scale, out=again)
    assert torch.equal(out, again), "the same call gives the same bits"


@DTYPES
@pytest.mark.parametrize("dim", [64, 65])
def test_accumulate(dim, dtype):
    tokens, rows = 500, 300
    ids, dy, old = make_ids(tokens, rows, "text"), normal(tokens, dim, dtype=BF16), normal(rows, dim, dtype=dtype, seed=2)
    want, room = embedding_backward64(dy, ids, rows, 2.0)
    out = old.cuda()
    ops.embedding_backward(dy.cuda(), ids.cuda(), rows, scale=2.0, out=out, accumulate=True)
    assert_near(out, want + old.double(), room + 2 * U32 * (want.abs() + old.double().abs()))
    unused = torch.ones(rows, dtype=torch.bool)
    unused[ids[(ids >= 0) & (ids < rows)]] = False
    assert unused.any() and torch.equal(out.cpu()[unused], old[unused])


@pytest.mark.parametrize("offset", [0, 8, 3])
def test_slices_of_flat_buffers(offset):
    # a table in the gathered unit buffer, its gradient in a replica's flat gradient
    tokens, rows, dim = 300, 40, 72
    ids, dy = make_ids(tokens, rows, "text"), normal(tokens, dim, dtype=BF16, seed=3)
    flat = normal(offset + rows * dim + 11, dtype=BF16, seed=4).cuda()
    grad = torch.full_like(flat, 7.0)
    spot = slice(offset, offset + rows * dim)
    table = flat[spot].view(rows, dim)
    got = ops.embedding(ids.cuda(), table)
    assert_near(got, looked_up(ids, table.cpu(), 1.0), 0.0)
    ops.embedding_backward(dy.cuda(), ids.cuda(), rows, out=grad[spot].view(rows, dim))
    assert_near(grad[spot].view(rows, dim), *embedding_backward64(dy, ids, rows, 1.0))
    grad[spot] = 7.0
    assert (grad == 7.0).all()


def test_strides_and_shapes():
    ids = make_ids(24, 30, "any").view(2, 3, 4)
    wide, dwide = normal(30, 50, dtype=BF16, seed=5).cuda(), normal(24, 90, dtype=BF16, seed=6).cuda()
    table = wide[:, 3:43]
    want = looked_up(ids, table.cpu(), 1.0)
    out = torch.full((2, 3, 4, 48), 5.0, dtype=BF16, device="cuda")
    ops.embedding(ids.cuda(), table, out=out[..., 8:])
    assert_near(out[..., 8:], want, 0.0)
    assert (out[..., :8] == 5.0).all()
    dy = dwide.view(2, 3, 4, 90)[..., 1:41]
    gradient, room = embedding_backward64(dy.cpu(), ids, 30, 1.0)
    into = torch.full((30, 44), 5.0, device="cuda")
    ops.embedding_backward(dy, ids.cuda(), 30, out=into[:, 2:42])
    assert_near(into[:, 2:42], gradient, room)
    assert (into[:, :2] == 5.0).all() and (into[:, 42:] == 5.0).all()
    turned = ids.transpose(0, 2).cuda()  # ids and a gradient whose strides fit no matrix
    assert torch.equal(ops.embedding(turned, table), ops.embedding(turned.contiguous(), table))
    assert_near(ops.embedding_backward(dy.transpose(0, 2), turned, 30, out=torch.empty(30, 40, device="cuda")), gradient, room)
    single = torch.tensor(4, device="cuda")
    assert torch.equal(ops.embedding(single, table), table[4])
    one = ops.embedding_backward(table[4], single, 30)
    assert torch.equal(one[4], table[4]) and one.count_nonzero() == one[4].count_nonzero()


def test_nothing():
    for dtype in (torch.int32, torch.int64):
        none, ids = torch.empty(0, dtype=dtype, device="cuda"), torch.tensor([0, 5, -1], dtype=dtype, device="cuda")
        table = torch.ones(6, 16, device="cuda")
        assert ops.embedding(none, table).shape == (0, 16)
        assert (ops.embedding_backward(torch.empty(0, 16, device="cuda"), none, 6) == 0).all()
        assert torch.equal(ops.embedding_backward(torch.empty(0, 16, device="cuda"), none, 6, out=table, accumulate=True), table)
        empty = torch.empty(0, 16, device="cuda")
        assert (ops.embedding(ids, empty) == 0).all()
        assert ops.embedding_backward(torch.ones(3, 16, device="cuda"), ids, 0).shape == (0, 16)
        padding = torch.full((70,), -1, dtype=dtype, device="cuda")
        poison = torch.full((70, 16), float("nan"), device="cuda")
        assert (ops.embedding_backward(poison, padding, 6) == 0).all(), "what is behind padding reaches no sum"


def test_not_finite():
    ids = torch.tensor([0, 1, 1, 2, 1, 0], device="cuda")
    dy = torch.ones(6, 40, device="cuda")
    dy[2, 3], dy[3, 5] = float("nan"), float("inf")
    got = ops.embedding_backward(dy, ids, 4)
    assert got[1, 3].isnan() and got[2, 5].isinf() and got.isfinite().sum() == 4 * 40 - 2


def test_streams_and_capture():
    ids, dy = make_ids(5000, 900, "text").cuda(), normal(5000, 128, dtype=BF16).cuda()
    table = normal(900, 128, dtype=BF16, seed=2).cuda()
    want, grad = ops.embedding(ids, table), ops.embedding_backward(dy, ids, 900)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = ops.embedding_backward(dy, ids, 900)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(other, grad)
    static, graph = torch.zeros_like(ids), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ops.embedding(static, table)
        g = ops.embedding_backward(dy, static, 900)
    for _ in range(2):
        static.copy_(ids)
        graph.replay()
        assert torch.equal(y, want) and torch.equal(g, grad)
        static.zero_()
        graph.replay()


def test_offsets_past_32_bits():
    rows, dim = (1 << 20) + 4, 2056
    table = torch.zeros(rows, dim, dtype=BF16, device="cuda")
    ids = torch.tensor([rows - 1, 0, rows - 2, rows - 1], device="cuda")
    table[rows - 1], table[rows - 2] = 2.0, 3.0
    got = ops.embedding(ids, table)
    assert (got[[0, 3]] == 2.0).all() and (got[1] == 0).all() and (got[2] == 3.0).all()
    table.fill_(9.0)
    dy = torch.ones(4, dim, dtype=BF16, device="cuda")
    ops.embedding_backward(dy, ids, rows, out=table)
    assert (table[rows - 1] == 2.0).all() and (table[rows - 2] == 1.0).all() and (table[0] == 1.0).all()
    assert float(table.sum(dtype=torch.float64)) == 4.0 * dim
    # the same of the looked up rows and their gradient
    tokens, dim = 39, 64
    stride = (1 << 31) // (tokens - 1) // 64 * 64 + 64
    big = table.view(-1)[:(tokens - 1) * stride + dim].as_strided((tokens, dim), (stride, 1))
    ids, dy = make_ids(tokens, 9, "text").cuda(), normal(tokens, dim, dtype=BF16).cuda()
    big.copy_(dy)
    assert torch.equal(ops.embedding_backward(big, ids, 9), ops.embedding_backward(dy, ids, 9))
    small = normal(9, dim, dtype=BF16).cuda()
    ops.embedding(ids, small, out=big)
    assert torch.equal(big, ops.embedding(ids, small))


def test_autograd():
    ids = make_ids(200, 30, "text").view(4, 50).cuda()
    table = normal(30, 48, seed=7).cuda().requires_grad_()
    dy = normal(200, 48, seed=8).view(4, 50, 48).cuda()
    y = ops.embedding_autograd(ids, table, scale=2.5)
    y.backward(dy)
    assert torch.equal(y, ops.embedding(ids, table.detach(), scale=2.5))
    assert torch.equal(table.grad, ops.embedding_backward(dy, ids, 30, scale=2.5))
    table.grad = None
    ops.embedding_autograd(ids, table).sum().backward()  # a gradient with strides of zero
    assert torch.equal(table.grad, ops.embedding_backward(torch.ones_like(dy), ids, 30))
    grads = torch.autograd.grad(ops.embedding_autograd(ids, table).square().sum(), table, create_graph=True)
    with pytest.raises(RuntimeError):
        (grads[0].square().sum() + table.square().sum()).backward()
    with pytest.raises(ValueError):
        ops.embedding(ids, table)
    with pytest.raises(ValueError):
        ops.embedding_backward(dy.requires_grad_(), ids, 30)


def test_gradient_against_differences():
    ids, dy = make_ids(90, 20, "text").cuda(), normal(90, 32, seed=9).cuda()
    table, direction = normal(20, 32, seed=10).cuda(), normal(20, 32, seed=11).cuda()
    grad = ops.embedding_backward(dy, ids, 20, scale=1.5)
    value = [float((ops.embedding(ids, table + sign * direction, scale=1.5).double() * dy).sum()) for sign in (1, -1)]
    want = float((grad.double() * direction).sum())
    # linear in the table: only fp32's roundings of a few thousand terms of order one
    assert abs((value[0] - value[1]) / 2 - want) <= 1e-3


def test_tensor_checks():
    ids, table = torch.tensor([0, 1, 2], device="cuda"), torch.ones(5, 16, device="cuda")
    dy = torch.ones(3, 16, device="cuda")
    for bad in (ids.short(), ids.float(), ids.cpu()):
        with pytest.raises(ValueError):
            ops.embedding(bad, table)
        with pytest.raises(ValueError):
            ops.embedding_backward(dy, bad, 5)
    for bad in (table.half(), table.cpu(), table.t(), table[0], table[:, :0]):
        with pytest.raises(ValueError):
            ops.embedding(ids, bad)
    for out in (dy[:2], dy.bfloat16(), table[:3], dy[:1].expand(3, 16)):
        with pytest.raises(ValueError):
            ops.embedding(ids, table, out=out)
    for bad in (dy[:2], dy.half(), dy.t(), dy[0]):
        with pytest.raises(ValueError):
            ops.embedding_backward(bad, ids, 5)
    for out in (table[:4], table.half(), table.t().contiguous().t(), dy, table[:1].expand(5, 16)):
        with pytest.raises(ValueError):
            ops.embedding_backward(dy, ids, 5, out=out)
    big = torch.ones(8, 16, device="cuda")
    with pytest.raises(ValueError):
        ops.embedding_backward(big[:3], ids, 5, out=big[2:7])
    with pytest.raises(ValueError):
        ops.embedding_backward(dy, ids, 5, accumulate=True)
    for bad in (-1, (1 << 30) + 1):
        with pytest.raises((B.ZeroError, RuntimeError)):
            ops.embedding_backward(dy, ids, bad, out=None)
    with pytest.raises(TypeError):
        ops.embedding_backward(dy, ids, 5.0)
