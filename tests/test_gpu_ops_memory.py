"""Outputs given by the caller: what may share memory with what."""

import pytest
import torch

from muon_reference import rotation_table
from zero_sharded_mixed_flatparameter_gb300 import binding as B
from zero_sharded_mixed_flatparameter_gb300 import ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_sharded_mixed_flatparameter_gb300 import build_lib
    build_lib.build()
    B.load()


def normal(*shape, dtype=torch.bfloat16):
    gen = torch.Generator(device="cuda").manual_seed(sum(shape))
    return torch.empty(shape, device="cuda").normal_(generator=gen).to(dtype)


def test_orthogonalize_refuses_overlaps():
    x = normal(3, 40, 50)
    for out in (x, x.flip(0).copy_(x)[:1].expand(3, 40, 50)):
        with pytest.raises(ValueError):
            ops.orthogonalize(x, out=out)
    wide = normal(40, 120)
    with pytest.raises(ValueError):
        ops.orthogonalize(wide[:, :60], out=wide[:, 59:119])
    want = ops.orthogonalize(wide[:, :60])
    assert torch.equal(ops.orthogonalize(wide[:, :60], out=wide[:, 60:]), want)


@pytest.mark.parametrize("dim,rotary", [(64, 64), (80, 32), (6, 4)])
def test_norm_and_rotation_outputs(dim, rotary):
    table = rotation_table(32, rotary).cuda()
    q, k, dq, dk = normal(9, 3, dim), normal(9, 2, dim), normal(9, 3, dim + 1)[..., :dim], normal(9, 2, dim)
    rest = (None, None, table)
    want, back = ops.qk_norm_rope(q, k, *rest), ops.qk_norm_rope_backward(dq, dk, q, k, *rest)
    for out in ((q, q[:, :2]), (torch.empty_like(q), q[:, :2]), (k[:, :1].expand(9, 3, dim), torch.empty_like(k)),
                (torch.empty_like(q), k[:1].expand(9, 2, dim))):
        with pytest.raises(ValueError):
            ops.qk_norm_rope(q, k, *rest, out=out)
        with pytest.raises(ValueError):
            ops.qk_norm_rope_backward(dq, dk, q, k, *rest, out=out)
    gains = torch.empty(dim + dim // 2, device="cuda")
    with pytest.raises(ValueError):
        ops.qk_norm_rope_backward(dq, dk, q, k, *rest, gain_out=(gains[:dim], gains[-dim:]))
    with pytest.raises(ValueError):
        ops.qk_norm_rope_backward(dq, dk, q, k, *rest, gain_out=(gains[:dim], gains[:dim]))
    # in place: onto the gradients, onto the queries and keys, and forward
    a, b = dq.clone(), dk.clone()
    for x, y in zip(ops.qk_norm_rope_backward(a, b, q, k, *rest, out=(a, b)), back):
        assert torch.equal(x, y)
    a, b = q.clone(), k.clone()
    for x, y in zip(ops.qk_norm_rope_backward(dq, dk, a, b, *rest, out=(a, b)), back):
        assert torch.equal(x, y)
    for x, y in zip(ops.qk_norm_rope(q, k, *rest, out=(q, k)), want):
        assert torch.equal(x, y)
