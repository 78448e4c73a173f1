"""Outputs that the caller gives to the layer norm, the 8-bit form and the
embedding: what they must not share, and what torch.autograd learns of them."""

import pytest
import torch

from zero_sharded_mixed_flatparameter_gb300 import binding as B
from zero_sharded_mixed_flatparameter_gb300 import ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_sharded_mixed_flatparameter_gb300 import build_lib
    build_lib.build()
    B.load()


def normal(*shape, seed=0):
    return torch.empty(shape, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(seed + sum(shape)))


def test_outputs_over_weights_and_statistics():
    rows, cols = 6, 64
    x, dy, w, b = normal(rows, cols), normal(rows, cols, seed=1), normal(cols), normal(cols, seed=1)
    want, stats, packed = ops.layer_norm(x, w, b, pack=torch.int8)
    buffer = normal(rows * cols + cols, seed=2)
    y = buffer[:rows * cols].view(rows, cols)
    over = buffer[3:3 + 2 * rows].view(rows, 2)
    over = over if over.data_ptr() % 8 == 0 else buffer[4:4 + 2 * rows].view(rows, 2)
    over.copy_(stats)
    before = buffer.clone()
    for at in (0, cols + 5, rows * cols - 1):
        vector = buffer[at:at + cols]
        for args in ((vector, None), (vector, b), (w, vector), (None, vector)):
            with pytest.raises(ValueError):
                ops.layer_norm(x, *args, out=y)
        for source in (x, packed):
            with pytest.raises(ValueError):
                ops.layer_norm_backward(dy, source, vector, stats, out=y)
    for source in (x, packed):
        with pytest.raises(ValueError):
            ops.layer_norm_backward(dy, source, w, over, out=y)
        with pytest.raises(ValueError):
            ops.layer_norm_backward(dy, source, None, over, out=y)
    assert torch.equal(buffer, before), "a refused call writes nothing"
    # beside them in one buffer
    beside = buffer[rows * cols:]
    beside.copy_(w)
    got, _ = ops.layer_norm(x, beside, b, out=y)
    assert torch.equal(got, want)
    for source in (x, packed):
        grads = ops.layer_norm_backward(dy, source, w, stats)
        for g, e in zip(ops.layer_norm_backward(dy, source, beside, stats, out=y), grads):
            assert torch.equal(g, e)


def test_norm_and_rotation_over_gains_table_and_positions():
    tokens, dim = 5, 32
    q, k, dq, dk = normal(tokens, 3, dim), normal(tokens, 2, dim), normal(tokens, 3, dim, seed=1), normal(tokens, 2, dim, seed=1)
    gains, table = (normal(dim), normal(dim, seed=1)), normal(8, 16).cos()
    positions = torch.arange(tokens, dtype=torch.int32, device="cuda")
    buffer = normal(q.numel() + 200, seed=2)
    out = (buffer[:q.numel()].view_as(q), torch.empty_like(k))
    before = buffer.clone()
    end = buffer[q.numel() - 1:]  # the last element of the one output and what is behind it
    for bad in ((end[:dim], gains[1], table, positions), (gains[0], end[:dim], table, positions),
                (None, None, end[:128].view(8, 16), positions), (*gains, table, end[:tokens].view(torch.int32))):
        with pytest.raises(ValueError):
            ops.qk_norm_rope(q, k, *bad, out=out)
        with pytest.raises(ValueError):
            ops.qk_norm_rope_backward(dq, dk, q, k, *bad, out=out)
    with pytest.raises(ValueError):  # one output over another
        ops.qk_norm_rope_backward(dq, dk, q, k, *gains, table, positions, out=out, gain_out=(end[:dim], torch.empty_like(gains[0])))
    assert torch.equal(buffer, before), "a refused call writes nothing"
    want = ops.qk_norm_rope_backward(dq, dk, q, k, *gains, table, positions)
    beside = (end[1:1 + dim], end[1 + dim:1 + 2 * dim])
    for g, e in zip(ops.qk_norm_rope_backward(dq, dk, q, k, *gains, table, positions, out=out, gain_out=beside), want):
        assert torch.equal(g, e)
    beside[0].copy_(gains[0])
    for g, e in zip(ops.qk_norm_rope(q, k, beside[0], gains[1], table, positions, out=out),
                    ops.qk_norm_rope(q, k, *gains, table, positions)):
        assert torch.equal(g, e)


def calls_with_outputs():
    """Every operator with outputs of the caller's: a function of a tuple of them, and their shapes."""
    x, dy, w, b = normal(6, 64), normal(6, 64, seed=1), normal(64), normal(64, seed=1)
    _, stats, packed = ops.layer_norm(x, w, b, pack=torch.int8)
    ids, table = torch.tensor([0, 2, 2], device="cuda"), normal(5, 16)
    q, k, dq, dk = normal(4, 3, 32), normal(4, 2, 32), normal(4, 3, 32, seed=1), normal(4, 2, 32, seed=1)
    rest = normal(32), normal(32, seed=1), normal(8, 16).cos()
    return [
        (lambda out: ops.layer_norm(x, w, b, out=out[0]), [(6, 64)]),
        (lambda out: ops.layer_norm_backward(dy, x, w, stats, out=out[0], weight_out=out[1], bias_out=out[2]), [(6, 64), (64,), (64,)]),
        (lambda out: ops.unpack_activations(packed, out=out[0]), [(6, 64)]),
        (lambda out: ops.embedding(ids, table, out=out[0]), [(3, 16)]),
        (lambda out: ops.embedding_backward(dy[:3, :16], ids, 5, out=out[0]), [(5, 16)]),
        (lambda out: ops.embedding_backward(dy[:3, :16], ids, 5, out=out[0], accumulate=True), [(5, 16)]),
        (lambda out: ops.qk_norm_rope(q, k, *rest, out=out), [q.shape, k.shape]),
        (lambda out: ops.qk_norm_rope_backward(dq, dk, q, k, *rest, out=out[:2], gain_out=out[2:]), [q.shape, k.shape, (32,), (32,)]),
        (lambda out: ops.orthogonalize(x, out=out[0]), [(6, 64)])]


@pytest.mark.parametrize("which", range(9))
def test_outputs_that_require_gradients(which):
    call, shapes = calls_with_outputs()[which]
    dtype = torch.bfloat16 if which == 8 else torch.float32
    for i in range(len(shapes)):
        outs = tuple(torch.zeros(s, device="cuda", dtype=dtype) for s in shapes)
        for leaf in (outs[i].clone().requires_grad_(), outs[i].clone().requires_grad_() * 1):
            some = (*outs[:i], leaf, *outs[i + 1:])
            with pytest.raises(ValueError):
                call(some)
            assert (leaf == 0).all()
            with torch.no_grad():  # as torch's own calls into a leaf
                call(some)
            assert not (leaf == 0).all()


@pytest.mark.parametrize("which", range(9))
def test_autograd_learns_of_what_is_written(which):
    call, shapes = calls_with_outputs()[which]
    dtype = torch.bfloat16 if which == 8 else torch.float32
    for i in range(len(shapes)):
        outs = tuple(torch.zeros(s, device="cuda", dtype=dtype) for s in shapes)
        versions = [o._version for o in outs]
        leaf = torch.ones_like(outs[i]).requires_grad_()
        product = leaf * outs[i]  # keeps outs[i] for the leaf's gradient
        call(outs)
        assert all(o._version > v for o, v in zip(outs, versions))
        with pytest.raises(RuntimeError):
            product.sum().backward()
    with torch.inference_mode():  # such tensors have no version
        call(tuple(torch.zeros(s, device="cuda", dtype=dtype) for s in shapes))


def test_autograd_learns_of_codes_written_again():
    x = normal(6, 64)
    packed = ops.pack_activations(x)
    version = packed.data._version
    ops.pack_activations(2 * x, out=packed)
    assert packed.data._version > version


def test_a_kept_input_that_changes_is_found():
    # the norm keeps x; a lookup into the same memory comes before its backward pass
    x, w = normal(3, 16), normal(16).requires_grad_()
    y = ops.layer_norm_autograd(x, w)
    ops.embedding(torch.tensor([1, 0, 1], device="cuda"), normal(2, 16, seed=3), out=x)
    with pytest.raises(RuntimeError):
        y.sum().backward()
