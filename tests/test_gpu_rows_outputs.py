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
