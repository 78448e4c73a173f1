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


def test_inputs_that_require_gradients():
    # a result cut from the graph would train nothing, silently
    leaves, table = inputs()
    plain = [x.detach() for x in leaves]
    x = torch.randn(8, 8, device="cuda", requires_grad=True)
    dq, dk = torch.randn_like(plain[0]), torch.randn_like(plain[1])
    with pytest.raises(ValueError):
        ops.orthogonalize(x)
    for i in range(4):
        args = list(plain)
        args[i] = leaves[i]
        with pytest.raises(ValueError):
            ops.qk_norm_rope(*args, table)
        with pytest.raises(ValueError):
            ops.qk_norm_rope_backward(dq, dk, *args, table)
    with pytest.raises(ValueError):
        ops.qk_norm_rope_backward(dq.requires_grad_(), dk, *plain, table)
    want = [*ops.qk_norm_rope(*plain, table), *ops.qk_norm_rope_backward(dq.detach(), dk, *plain, table)]
    with torch.no_grad():
        assert torch.equal(ops.orthogonalize(x), ops.orthogonalize(x.detach()))
        got = [*ops.qk_norm_rope(*leaves, table), *ops.qk_norm_rope_backward(dq, dk, *leaves, table)]
    for a, b in zip(got, want):
        assert torch.equal(a, b) and not a.requires_grad
