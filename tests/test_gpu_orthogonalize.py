"""Newton-Schulz orthogonalisation on the GPU against 64 bits."""

import pytest
import torch

from muon_reference import NS_TOL, orthogonalized64, relative
from zero_sharded_mixed_flatparameter_gb300 import binding as B
from zero_sharded_mixed_flatparameter_gb300 import ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_sharded_mixed_flatparameter_gb300 import build_lib
    build_lib.build()
    B.load()


def normal(shape, seed, std=1e-3):
    return torch.empty(shape).normal_(0.0, std, generator=torch.Generator().manual_seed(seed))


SHAPES = [(1, 1), (1, 7), (7, 1), (2, 3), (16, 16), (33, 17), (64, 64), (64, 130), (127, 129), (128, 128), (130, 64),
          (128, 1024), (129, 257), (257, 129), (255, 640), (640, 255), (256, 2000), (2000, 256), (384, 384),
          (513, 777), (777, 513), (1, 5000), (5000, 1), (8, 4096), (300, 4100), (150, 6000), (6000, 150), (130, 1100),
          (400, 2100), (2100, 400), (640, 1500)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_against_64_bits(rows, cols, dtype):
    x = normal((rows, cols), rows * 10007 + cols).to(dtype)
    got = ops.orthogonalize(x.cuda())
    assert got.dtype == torch.bfloat16 and got.shape == x.shape
    assert relative(got, orthogonalized64(x)) <= NS_TOL


@pytest.mark.parametrize("rows,cols", [(8, 300), (128, 129), (129, 128), (100, 3000), (3000, 100), (120, 257), (17, 520),
                                       (1025, 33), (2, 20000), (70, 2100), (2100, 70), (9, 4000), (128, 5000)])
@pytest.mark.parametrize("rank", [0, 1, 3])
def test_thin_matrices_are_nearly_exact(rows, cols, rank):
    # Thin matrices keep 22 bits throughout: what is left is the bf16 result,
    # rms 2^-9 / sqrt(3) = 1.1e-3 of it over many elements and at most 2^-8 / 2,
    # and up to 4e-4 for a low rank.
    x = normal((rows, cols), rows + cols, 1.0)
    if rank:
        x = normal((rows, rank), 3, 1.0) @ normal((rank, cols), 4, 1.0)
    want = orthogonalized64(x)
    assert relative(ops.orthogonalize(x.cuda()), want) <= 2.5e-3


@pytest.mark.parametrize("batch,rows,cols", [(2112, 1040, 1010), (250000, 64, 136)])
def test_stack_of_more_than_2_to_the_31_elements(batch, rows, cols):
    x = normal((rows, cols), batch).cuda()
    got = ops.orthogonalize(x.expand(batch, rows, cols))
    assert got.numel() > 2 ** 31
    assert relative(got[batch - 1], orthogonalized64(x.cpu())) <= NS_TOL
    assert all(torch.equal(part, got[:1].expand_as(part)) for part in got.split(batch // 16 + 1))


@pytest.mark.parametrize("batch,rows,cols", [(3, 65, 40), (5, 40, 65), (2, 300, 520), (9, 128, 128), (70, 24, 9),
                                             (70, 130, 140)])
def test_stack(batch, rows, cols):
    x = normal((batch, rows, cols), batch)
    x[1] *= 1e4  # the scale of one matrix is its own affair
    got = ops.orthogonalize(x.cuda())
    for i in range(batch):
        assert relative(got[i], orthogonalized64(x[i])) <= NS_TOL, i
    alone = ops.orthogonalize(x[batch - 1].cuda())
    assert torch.equal(alone, got[batch - 1]), "a matrix does not depend on its neighbours"


@pytest.mark.parametrize("rank", [1, 2, 8])
@pytest.mark.parametrize("rows,cols", [(96, 96), (200, 700), (700, 200)])
def test_low_rank(rows, cols, rank):
    # the part outside the rank is noise of the rounding; it must not be blown up
    x = normal((rows, rank), 3, 1.0) @ normal((rank, cols), 4, 1.0)
    assert relative(ops.orthogonalize(x.cuda()), orthogonalized64(x)) <= NS_TOL


@pytest.mark.parametrize("rows,cols", [(150, 150), (96, 500)])
def test_decaying_spectrum(rows, cols):
    m = min(rows, cols)
    u, v = torch.linalg.qr(normal((rows, m), 5, 1.0))[0], torch.linalg.qr(normal((cols, m), 6, 1.0))[0]
    x = (u * torch.logspace(0, -4, m)) @ v.T
    assert relative(ops.orthogonalize(x.cuda()), orthogonalized64(x)) <= NS_TOL


@pytest.mark.parametrize("steps", [1, 2, 3, 7])
@pytest.mark.parametrize("coefficients", [(3.4445, -4.7750, 2.0315), (1.5, -0.5, 0.0), (15 / 8, -10 / 8, 3 / 8)])
def test_steps_and_coefficients(steps, coefficients):
    for shape in ((90, 140), (140, 90)):
        x = normal(shape, steps)
        want = orthogonalized64(x, steps, coefficients)
        assert relative(ops.orthogonalize(x.cuda(), steps=steps, coefficients=coefficients), want) <= NS_TOL


def test_strides_and_out():
    big = normal((4, 70, 211), 8).cuda()
    x = big[::2, 1::3, 5:100]
    out = torch.full((2, 23, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    view = out[:, :, 7:102]
    assert ops.orthogonalize(x, out=view) is view
    for i in range(2):
        assert relative(view[i], orthogonalized64(x[i].cpu())) <= NS_TOL
    assert out[:, :, :7].isnan().all() and out[:, :, 102:].isnan().all(), "only the view is written"


def test_expanded_input():
    x = normal((40, 33), 9).cuda()
    got = ops.orthogonalize(x.expand(3, 40, 33))
    assert torch.equal(got[0], got[2]) and relative(got[1], orthogonalized64(x.cpu())) <= NS_TOL


@pytest.mark.parametrize("shape", [(64, 64), (300, 200), (130, 513)])
def test_zero_matrix_and_nonfinite(shape):
    x = torch.zeros((3, *shape))
    x[1] = normal(shape, 10)
    assert (ops.orthogonalize(x.cuda())[0] == 0).all()
    x[0] = x[1]
    x[0, 3, 5] = float("inf")
    x[2] = x[1]
    x[2, 0, 1] = float("nan")
    got = ops.orthogonalize(x.cuda())
    assert got[0].isnan().all() and got[2].isnan().all()
    assert relative(got[1], orthogonalized64(x[1])) <= NS_TOL


def test_extreme_magnitudes():
    for scale in (1e-15, 1e12):
        x = normal((120, 77), 11, 1.0) * scale
        assert relative(ops.orthogonalize(x.cuda(), eps=0.0), orthogonalized64(x, eps=0.0)) <= NS_TOL


def test_one_large_row():
    x = normal((100, 300), 12)
    x[17] *= 1e3
    x[40:] = 0
    assert relative(ops.orthogonalize(x.cuda()), orthogonalized64(x)) <= NS_TOL


@pytest.mark.parametrize("shape", [(0, 5), (5, 0), (0, 4, 4), (2, 0, 3)])
def test_empty(shape):
    assert ops.orthogonalize(torch.empty(shape, device="cuda")).shape == shape


def test_reproducible_and_other_stream():
    x = normal((2, 333, 450), 13).cuda()
    first = ops.orthogonalize(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        second = ops.orthogonalize(x)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(first, second)


def test_captured():
    x = normal((257, 130), 14).cuda()
    want = ops.orthogonalize(x)
    out = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.orthogonalize(x, out=out)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def call(rows=8, cols=8, batch=1, cfg=None, **over):
    x = torch.zeros(1 << 17, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    a = dict(src=x.data_ptr(), in_dtype=B.ZERO_GRAD_FP32, in_row_stride=cols, in_batch_stride=rows * cols,
             out=x.data_ptr() + (1 << 18), out_row_stride=cols, out_batch_stride=rows * cols, workspace=ws.data_ptr(),
             workspace_bytes=1 << 20)
    a.update(over)
    B.zero_orthogonalize(cfg or B.make_ns_config(), rows, cols, batch, *a.values())
    torch.cuda.synchronize()


@pytest.mark.parametrize("over", [
    dict(src=0), dict(out=0), dict(in_row_stride=7),
    dict(rows=136, cols=136, workspace=0), dict(rows=136, cols=136, workspace_bytes=1000),
    dict(out_row_stride=7), dict(in_dtype=2), dict(rows=-1), dict(batch=-1), dict(in_batch_stride=-1),
    dict(batch=2, out_batch_stride=63), dict(cfg=B.zero_ns_config(0, 1.5, -0.5, 0.0, 0.0)),
    dict(cfg=B.zero_ns_config(5, float("nan"), 0.0, 0.0, 0.0)), dict(cfg=B.zero_ns_config(5, 1.5, -0.5, 0.0, -1.0)),
    dict(cfg=B.zero_ns_config(5, 30.0, 1.0, 1.0, 0.0)),
], ids=str)
def test_refusals(over):
    call(**{k: v for k, v in over.items() if v == 136})
    with pytest.raises(B.ZeroError) as e:
        call(**over)
    assert e.value.status == B.ZERO_EINVAL


def test_misaligned_pointers():
    x = torch.zeros(4096, device="cuda").data_ptr()
    for over in (dict(src=x + 2), dict(out=x + 1), dict(rows=136, cols=136, workspace=x + 16)):
        with pytest.raises(B.ZeroError) as e:
            call(**over)
        assert e.value.status == B.ZERO_EINVAL


def test_host_pointer():
    host = torch.zeros(64)
    with pytest.raises(B.ZeroError) as e:
        call(src=host.data_ptr())
    assert e.value.status == B.ZERO_EINVAL


def test_tensor_checks():
    good = torch.zeros(8, 8, device="cuda")
    for bad in (torch.zeros(8, device="cuda"), torch.zeros(8, 8), good.half(), good.t()[:, ::2]):
        with pytest.raises(ValueError):
            ops.orthogonalize(bad)
    with pytest.raises(ValueError):
        ops.orthogonalize(good, out=good)
