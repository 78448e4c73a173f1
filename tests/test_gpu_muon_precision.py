"""The precision that the orthogonalisation promises, over the steps it promises it for."""

import math

import pytest
import torch

from muon_reference import orthogonalized64, relative
from test_gpu_orthogonalize import normal
from zero_sharded_mixed_flatparameter_gb300 import binding as B
from zero_sharded_mixed_flatparameter_gb300 import ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_sharded_mixed_flatparameter_gb300 import build_lib
    build_lib.build()
    B.load()


def tolerance(steps):
    # three roundings of 2^-11 / sqrt(3) a step, each passing polynomials of a
    # relative slope below 4, in quadrature; the bf16 result adds 2^-9
    return 2.0 ** -11 / math.sqrt(3) * math.sqrt(3 * steps) * 4 + 2.0 ** -9


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("rank", [1, 2, 8, 40, None])
@pytest.mark.parametrize("rows,cols", [(200, 700), (700, 200), (300, 300), (96, 500)])
def test_any_rank_up_to_eight_steps(rows, cols, rank, steps):
    x = normal((rows, rank), 3, 1.0) @ normal((rank, cols), 4, 1.0) if rank else normal((rows, cols), 5)
    assert relative(ops.orthogonalize(x.cuda(), steps=steps), orthogonalized64(x, steps)) <= tolerance(steps)


@pytest.mark.parametrize("rows,cols", [(200, 700), (300, 300)])
def test_noise_outside_a_low_rank_stays_below_that_of_fp32(rows, cols):
    # ten steps: the noise has grown, in fp32 as well
    x = normal((rows, 1), 3, 1.0) @ normal((1, cols), 4, 1.0)
    want = orthogonalized64(x, 10)
    y = x / x.norm()
    for _ in range(10):
        s = y @ y.T
        y = 3.4445 * y + (-4.7750 * s + 2.0315 * (s @ s)) @ y
    assert relative(ops.orthogonalize(x.cuda(), steps=10), want) <= 4 * max(relative(y, want), tolerance(10))


@pytest.mark.parametrize("steps", [1, 2])
def test_larger_leading_coefficients(steps):
    coefficients = (8.28721201814563, -23.595886519098837, 17.300387312530933)
    for shape in ((200, 700), (300, 300)):
        x = normal((shape[0], 1), 3, 1.0) @ normal((1, shape[1]), 4, 1.0)
        got = ops.orthogonalize(x.cuda(), steps=steps, coefficients=coefficients)
        assert relative(got, orthogonalized64(x, steps, coefficients)) <= tolerance(steps)
