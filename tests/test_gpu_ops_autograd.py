"""How the operators meet torch.autograd."""

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


def inputs(grad=True):
    gen = torch.Generator(device="cuda").manual_seed(3)

    def normal(*shape):
        return torch.empty(shape, device="cuda").normal_(generator=gen).requires_grad_(grad)

    return [normal(6, 2, 64), normal(6, 1, 64), normal(64), normal(64)], rotation_table(16, 64).cuda()


def test_second_derivatives_are_refused():
    leaves, table = inputs()
    q, k = ops.qk_norm_rope_autograd(*leaves, table)
    grads = torch.autograd.grad(q.square().sum() + k.square().sum(), leaves, create_graph=True)
    # a penalty on the gradients that also depends on the inputs directly
    loss = sum(g.square().sum() for g in grads) + leaves[0].square().sum()
    with pytest.raises(RuntimeError):
        loss.backward()


def test_first_derivatives_repeat():
    leaves, table = inputs()
    for _ in range(2):
        q, k = ops.qk_norm_rope_autograd(*leaves, table)
        (q.square().sum() + k.sum()).backward()
    once = [x.grad / 2 for x in leaves]
    for x in leaves:
        x.grad = None
    q, k = ops.qk_norm_rope_autograd(*leaves, table)
    (q.square().sum() + k.sum()).backward()
    for x, g in zip(leaves, once):
        assert torch.equal(x.grad, g)
