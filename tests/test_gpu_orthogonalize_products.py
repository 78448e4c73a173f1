"""Newton-Schulz orthogonalisation with both sides above 128: what the thin form is tested for."""

import pytest
import torch

from muon_reference import NS_TOL, orthogonalized64, relative
from test_gpu_muon_precision import tolerance
from test_gpu_orthogonalize import normal
from zero_sharded_mixed_flatparameter_gb300 import binding as B
from zero_sharded_mixed_flatparameter_gb300 import ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_sharded_mixed_flatparameter_gb300 import build_lib
    build_lib.build()
    B.load()


@pytest.mark.parametrize("steps", [1, 2, 3, 7])
@pytest.mark.parametrize("coefficients", [(3.4445, -4.7750, 2.0315), (1.5, -0.5, 0.0), (15 / 8, -10 / 8, 3 / 8)])
def test_steps_and_coefficients(steps, coefficients):
    for shape in ((190, 340), (340, 190), (1100, 1200)):
        x = normal(shape, steps)
        want = orthogonalized64(x, steps, coefficients)
        assert relative(ops.orthogonalize(x.cuda(), steps=steps, coefficients=coefficients), want) <= tolerance(steps)


# by clusters of two, four and eight (alone, in stacks), by pairs of SMs, and singles
@pytest.mark.parametrize("batch,rows,cols", [(1, 1024, 1024), (1, 1100, 1200), (1, 1200, 1100), (4, 512, 2048), (2, 512, 2048),
                                             (1, 512, 2048), (1, 2048, 512), (8, 512, 2048), (2, 2048, 2100), (3, 777, 1301)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_forms(batch, rows, cols, dtype):
    x = normal((batch, rows, cols), rows + batch).to(dtype).cuda()
    got = ops.orthogonalize(x)
    for i in range(batch):
        assert relative(got[i], orthogonalized64(x[i])) <= NS_TOL, i
    assert torch.equal(ops.orthogonalize(x), got), "equal inputs give equal bits"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_strides_and_out(dtype):
    big = normal((4, 460, 411), 8).to(dtype).cuda()
    x = big[::2, 1::3, 5:305]
    out = torch.full((2, 153, 340), float("nan"), dtype=torch.bfloat16, device="cuda")
    view = out[:, :, 7:307]
    assert ops.orthogonalize(x, out=view) is view
    for i in range(2):
        assert relative(view[i], orthogonalized64(x[i].cpu())) <= NS_TOL
    assert out[:, :, :7].isnan().all() and out[:, :, 307:].isnan().all(), "only the view is written"


def test_expanded_input():
    x = normal((240, 233), 9).cuda()
    got = ops.orthogonalize(x.expand(3, 240, 233))
    assert torch.equal(got[0], got[2]) and relative(got[1], orthogonalized64(x.cpu())) <= NS_TOL


@pytest.mark.parametrize("shape", [(512, 2048), (1024, 1024), (2048, 2100)])
def test_nonfinite(shape):
    # in every form a matrix's NaN stays its own
    x = torch.stack([normal(shape, 2)] * 2)
    x[0, 7, 11] = float("inf")
    got = ops.orthogonalize(x.cuda())
    assert got[0].isnan().all() and relative(got[1], orthogonalized64(x[1])) <= NS_TOL
    alone = normal(shape, 2)
    alone[100, 200] = float("nan")
    assert ops.orthogonalize(alone.cuda()).isnan().all()


@pytest.mark.parametrize("batch,rows,cols", [(1, 512, 2048), (2, 512, 2048), (4, 2048, 512), (8, 512, 2048), (3, 777, 1301),
                                             (2, 2048, 2100), (9, 128, 700)])
def test_neighbours_values_do_not_count(batch, rows, cols):
    x = normal((batch, rows, cols), 4).cuda()
    got = ops.orthogonalize(x)[batch - 1]
    y = x.clone()
    y[:batch - 1] = normal((batch - 1, rows, cols), 5).cuda() * 1e5
    if batch > 1:
        y[0, 3, 4] = float("nan")
    assert torch.equal(ops.orthogonalize(y)[batch - 1], got)


def test_thin_matrices_are_the_same_in_any_stack():
    for shape in ((100, 700), (3000, 90), (64, 64)):
        x = normal((40, *shape), 6).cuda()
        want = ops.orthogonalize(x)
        for count in (1, 2, 7):
            assert torch.equal(ops.orthogonalize(x[:count]), want[:count])
