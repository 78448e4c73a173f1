"""Norms at the ends of the range, in the orthogonalisation and the Muon step."""

import numpy as np
import pytest
import torch

from muon_reference import NS_TOL, muon_scale, orthogonalized64, relative
from test_gpu_muon import LR, MU, WD, grads_for, make, mlp, reduced, snapshot, step
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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-24, 1e-12, 1e16, 1e25, 1e37])
@pytest.mark.parametrize("shape", SHAPES)
def test_any_finite_magnitude(shape, scale, dtype):
    x = (normal(shape, 3, 1.0) * scale).to(dtype)
    assert relative(ops.orthogonalize(x.cuda(), eps=0.0), orthogonalized64(x, eps=0.0)) <= NS_TOL
    # an eps of the norm's size still counts
    eps = min(float(x.double().norm()), 3e38)
    assert relative(ops.orthogonalize(x.cuda(), eps=eps), orthogonalized64(x, eps=float(np.float32(eps)))) <= NS_TOL


@pytest.mark.parametrize("shape", SHAPES)
def test_magnitudes_side_by_side(shape):
    # entries whose squares overflow beside ones whose squares underflow, row by row and matrix by matrix
    x = torch.stack([normal(shape, 5, 1.0)] * 4)
    x[0, ::2] *= 1e25
    x[1, 1::2] *= 1e-25
    x[2] *= 1e-25
    got = ops.orthogonalize(x.cuda(), eps=0.0)
    for i in range(4):
        assert relative(got[i], orthogonalized64(x[i], eps=0.0)) <= NS_TOL, i


@pytest.mark.parametrize("scale", [1e-25, 1e25])
@pytest.mark.parametrize("widths", [[16, 48, 16], [150, 300, 140], [30, 2000]])
def test_step_at_any_magnitude(widths, scale):
    pl, shapes = mlp(widths)
    fs = make(pl, shapes, 3, dtype="fp32", eps=0.0)
    grads = [g * (100 * scale) for g in grads_for(fs, pl, 3, "fp32", 1)]
    w0, g = fs.master.cpu().clone(), reduced(grads)
    step(fs, grads)
    for p, s in enumerate(shapes):
        if s is not None:
            at = slice(fs.param_offset(p), fs.param_offset(p) + pl.numel[p])
            assert torch.equal(fs.exp_avg.cpu()[at], g[at]), p
            want = orthogonalized64((g[at] + torch.tensor(MU) * g[at]).view(s), eps=0.0)
            size = LR * muon_scale(*s, "rms")
            update = (w0[at].double() * (1 - LR * WD) - fs.master.cpu()[at].double()) / size
            slack = float(w0[at].abs().max()) * 2.0 ** -22 / size * np.sqrt(want.numel()) / float(want.norm())
            assert relative(update.view(s), want) <= NS_TOL + slack, p


def test_long_sum():
    # 2^27 equal entries: added one after another in fp32, the last half of a
    # thread's 2^20 squares of 1.0153 would each lose a part to the sum's rounding
    n = 1 << 27
    x = torch.full((1, n), 1.0153, device="cuda")
    got = ops.orthogonalize(x, steps=1, coefficients=(1.0, 0.0, 0.0))
    want = torch.tensor(1 / np.sqrt(n), dtype=torch.float64).bfloat16()
    assert torch.equal(got, want.to(got.device).expand_as(got))
