"""Layer norm, 8-bit form and embedding gradient at the sizes of a training
batch: every thread takes several turns, with several real rows in flight, its
places in shared memory are used again and again, several groups of a CTA join
their column sums, and runs of sorted tokens are as long as they get.

Turns are counted for 152 SMs.  Tolerances are derived beside the plain forms in
rows_reference.py; what depends on the sizes is derived here.  The 64-bit forms
run on the GPU, in elementary operations."""

import pytest
import torch

from rows_reference import (E4M3, INT8, U32, assert_near, embedding_backward64_many, moments64, norm64, norm_backward64,
                            pack64_many)
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


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(*shape, seed, dtype=FP32):
    return torch.empty(shape, device="cuda").normal_(generator=generator(seed + sum(shape))).to(dtype)


def near(got, want, room):
    assert_near(got.reshape(want.shape), want.cpu(), room.cpu() if isinstance(room, torch.Tensor) else room)


# rows, columns: turns of the forward pass (bf16, fp32) and of the backward pass
NORMS = [
    (70001, 40),    # 8 lanes a row: 2.4; 2.4
    (40007, 128),   # 16 lanes a row: 2.7; 2.7
    (38011, 256),   # a warp a row, 4 rows in flight: 3.1, 3.1; 7.8, 7.8
    (38011, 264),   # 3.1, 6.3; 7.8, 15.6
    (15013, 1024),  # 2.5, 4.9; 6.2, 12.3
    (9500, 2048),   # 3.1, 6.3; 7.8, 15.6
    (2003, 4104),   # groups of three warps and of nine: 2.2, 2.2; 6.6, 13.2
    (1603, 8192),   # 2.1, 5.3; 5.3, 10.5
    (30011, 77),    # single elements: 2.5; 6.2
    (5003, 1301),   # groups of three warps: 2.7; 6.6
    (2503, 2047),   # 2.1 (groups of four warps); 4.1
    (1003, 8191),   # 3.3 (sixteen warps a row); 6.6
    (1300, 8200),   # rows that no CTA holds: 2.1; 2.1
]


@DTYPES
@pytest.mark.parametrize("center", [True, False], ids=["layer", "rms"])
@pytest.mark.parametrize("rows,cols", NORMS)
def test_layer_norm(rows, cols, center, dtype):
    """Means: at most 64 columns of a thread, 5 exchanges and 16 warps in a row,
    half of the columns in packed chains: below the 45 additions of norm64's room.
    Column sums: a thread adds at most 70001 / (456 * 32) < 5 (8 lanes a row), 38011 /
    (152 * 16) < 16 (a warp) or 1603 / 152 < 11 (a CTA) rows, then up to 16 groups,
    then 15 parts a warp and 32 warps: below the 128 additions of norm_backward64's
    room; rows that no CTA holds 1300 / 32 < 41, then 32 parts."""
    x = normal(rows, cols, seed=1) * (0.5 + normal(rows, 1, seed=2).abs()) + 0.3
    x[:, 3::97] *= 30  # a few columns far larger than the others
    x, dy = x.to(dtype), normal(rows, cols, seed=3, dtype=dtype)
    weight, bias = 1 + 0.2 * normal(cols, seed=4), 0.2 * normal(cols, seed=5)
    form = E4M3 if (rows + cols + center) % 2 else INT8
    y, stats, packed = ops.layer_norm(x, weight, bias, center=center, pack=form)
    near(y, *norm64(x, weight, bias, 1e-5, center))
    mean, rstd = moments64(x, 1e-5, center)
    near(stats[:, :1], mean, 48 * U32 * x.double().abs().mean(1, keepdim=True))
    near(stats[:, 1:], rstd, 64 * U32 * rstd)
    plain = ops.layer_norm(x, weight, bias, center=center)
    assert torch.equal(y, plain[0]) and torch.equal(stats, plain[1])
    codes, exponents, values = pack64_many(x, form)
    assert torch.equal(packed.codes.double(), codes) if form == INT8 else torch.equal(packed.codes.float().double(), codes)
    assert torch.equal(packed.scales.long(), exponents + 127)
    for kept, entries in ((x, x), (packed, values)):
        want = norm_backward64(dy, entries, weight, stats, center)
        got = ops.layer_norm_backward(dy, kept, weight, stats, center=center)
        for g, w in zip(got, want):
            near(g, *w)
        alone = ops.layer_norm_backward(dy, kept, weight, stats, center=center, bias=False)
        assert alone[2] is None and torch.equal(alone[0], got[0]) and torch.equal(alone[1], got[1])
        over = dy.clone()  # onto the gradient itself, later rows of which are on their way to shared memory
        again = ops.layer_norm_backward(over, kept, weight, stats, center=center, out=over)
        for g, w in zip(again, got):
            assert torch.equal(g, w), "the same call gives the same bits"


@FORMS
@DTYPES
@pytest.mark.parametrize("rows,cols", [
    (200003, 40),  # 8 lanes a row, four rows in flight: 2.1 turns
    (13001, 1000),  # 2.1
    (4001, 5000),  # a CTA walks over a row: 1.3
    (7003, 2048),  # 2.3
    (9001, 777),   # single elements: 3.0, back 5.9
    (60007, 31),   # 2.5, back 4.9
    (2003, 4999)])  # 1.3, back 2.6
def test_pack(rows, cols, dtype, form):
    x = (normal(rows, cols, seed=6) * normal(rows, cols, seed=7).mul_(3).exp_()).to(dtype)
    x[rows // 2, cols // 2], x[rows - 1, 0] = float("inf"), float("nan")
    packed = ops.pack_activations(x, form)
    codes, exponents, values = pack64_many(x, form)
    assert torch.equal(packed.codes.float().double(), codes)
    assert torch.equal(packed.scales.long(), exponents + 127)
    for out in (FP32, BF16):
        assert torch.equal(ops.unpack_activations(packed, out).nan_to_num(12345.0), values.to(out).nan_to_num(12345.0))


def ids_of(tokens, rows, kind):
    g = generator(tokens + rows)
    if kind == "text":  # the probability falls as 1 / id
        edge = torch.log(torch.tensor(rows + 1.0, dtype=torch.float64))
        ids = (torch.rand(tokens, generator=g, device="cuda", dtype=torch.float64) * edge.cuda()).exp().long() - 1
        ids.clamp_(0, rows - 1)
    elif kind == "one":
        return torch.full((tokens,), rows // 2, device="cuda")
    else:
        ids = torch.randint(0, rows, (tokens,), generator=g, device="cuda")
    ids[tokens // 3], ids[tokens - 1], ids[0] = -1, rows, 1 << 32
    return ids


@pytest.mark.parametrize("out_dtype", [FP32, BF16], ids=["out_fp32", "out_bf16"])
@DTYPES
@pytest.mark.parametrize("tokens,rows,dim,kind", [
    # runs of 32 tokens; about 50 tokens a row, so that rows reach up to 63 entries beyond a run's first 32
    (20011, 400, 2048, "any"), (20011, 400, 2047, "any"), (20011, 700, 2056, "any"), (160003, 3000, 8, "any"),
    (160003, 3000, 7, "any"), (40009, 900, 264, "any"), (40009, 900, 321, "any"),
    # frequent rows in many parts, others of a token; rows without tokens
    (20011, 30000, 2048, "text"), (40009, 70000, 263, "text"), (25013, 5, 1536, "text"), (160003, 160000, 9, "text"),
    (20011, 3, 2048, "one"), (160003, 2, 12, "one"),
    # runs of 16
    (12007, 300, 2048, "any"), (12007, 20000, 2047, "text"), (90001, 2000, 8, "any"), (25013, 600, 257, "any")])
def test_embedding_gradient(tokens, rows, dim, kind, dtype, out_dtype):
    ids, dy = ids_of(tokens, rows, kind), normal(tokens, dim, seed=8, dtype=dtype)
    want, room = embedding_backward64_many(dy, ids, rows, 1.5)
    out = torch.full((rows, dim), float("nan"), dtype=out_dtype, device="cuda")
    ops.embedding_backward(dy, ids, rows, scale=1.5, out=out)
    near(out, want, room)
    again = torch.empty_like(out)
    narrow = torch.where(ids == 1 << 32, -2, ids).int()  # no row, either
    ops.embedding_backward(dy, narrow, rows, scale=1.5, out=again)
    assert torch.equal(out, again), "the same call gives the same bits"
    old = normal(rows, dim, seed=9, dtype=out_dtype)
    both = old.clone()
    ops.embedding_backward(dy, ids, rows, scale=1.5, out=both, accumulate=True)
    near(both, want + old.double(), room + 2 * U32 * (want.abs() + old.double().abs()))
