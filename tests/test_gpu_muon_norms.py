"""Norms at the ends of the range, in the orthogonalisation and the Muon step."""

import numpy as np
import pytest
import torch

from muon_reference import NS_TOL, orthogonalized64, relative
from test_gpu_muon import LR, WD, make, mlp, snapshot, step
from test_gpu_orthogonalize import normal
from zero_sharded_mixed_flatparameter_gb300 import binding as B
from zero_sharded_mixed_flatparameter_gb300 import ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_sharded_mixed_flatparameter_gb300 import build_lib
    build_lib.build()
    B.load()


# one slice, many slices of a cluster, products alone and as a stack of tall ones
SHAPES = [(64, 64), (30, 2000), (2000, 30), (300, 200), (200, 1500)]


@pytest.mark.parametrize("eps", [0.0, 1e-7])
@pytest.mark.parametrize("shape", SHAPES)
def test_zero_matrix(shape, eps):
    x = torch.zeros((2, *shape))
    x[1] = normal(shape, 1)
    got = ops.orthogonalize(x.cuda(), eps=eps)
    assert (got[0] == 0).all()
    assert relative(got[1], orthogonalized64(x[1], eps=eps)) <= NS_TOL


@pytest.mark.parametrize("widths", [[16, 48, 16], [150, 300, 140], [30, 2000]])
def test_step_without_gradient_or_eps(widths):
    pl, shapes = mlp(widths)
    fs = make(pl, shapes, 2, eps=0.0)
    zero = [torch.zeros(fs.padded, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    before = snapshot(fs)
    step(fs, zero)
    decay = torch.tensor(1 - np.float64(np.float32(LR)) * np.float64(np.float32(WD)), dtype=torch.float64).float()
    for p, s in enumerate(shapes):
        if s is not None:
            at = slice(fs.param_offset(p), fs.param_offset(p) + pl.numel[p])
            assert torch.equal(fs.master.cpu()[at], before[0][at] * decay), p
            assert torch.equal(fs.param16.cpu()[at], (before[0][at] * decay).bfloat16()), p
