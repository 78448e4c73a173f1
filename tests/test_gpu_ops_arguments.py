"""Numbers given as something else than Python numbers."""

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


def test_an_eps_that_changes_in_place():
    q, k = torch.randn(5, 2, 64, device="cuda"), torch.randn(5, 1, 64, device="cuda")
    table, eps = rotation_table(8, 64).cuda(), torch.tensor(1e-6)
    for value in (1e-6, 10.0):
        eps.fill_(value)
        got = ops.qk_norm_rope(q, k, None, None, table, eps=eps)
        want = ops.qk_norm_rope(q, k, None, None, table, eps=value)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), value


def test_coefficients_that_change_in_place():
    x = torch.randn(40, 50, device="cuda")
    coefficients, eps = torch.tensor([3.4445, -4.7750, 2.0315], dtype=torch.float64), torch.tensor(0.0)
    first = ops.orthogonalize(x, coefficients=coefficients, eps=eps)
    assert torch.equal(first, ops.orthogonalize(x, eps=0.0))
    coefficients.copy_(torch.tensor([1.5, -0.5, 0.0]))
    eps.fill_(5.0)
    again = ops.orthogonalize(x, coefficients=coefficients, eps=eps)
    assert torch.equal(again, ops.orthogonalize(x, coefficients=(1.5, -0.5, 0.0), eps=5.0))
    assert not torch.equal(again, first)


def test_steps_are_whole():
    with pytest.raises(TypeError):
        ops.orthogonalize(torch.zeros(4, 4, device="cuda"), steps=5.5)


def test_waits_that_gave_up_are_counted_for_the_operators():
    before = ops.kernel_timeouts()
    for shape in ((64, 64), (30, 2000), (300, 200), (512, 2048)):
        ops.orthogonalize(torch.randn(shape, device="cuda"))
    assert ops.kernel_timeouts() == before == B.zero_kernel_timeouts()
    assert ops.kernel_timeouts("cuda:0") == before


def test_current_stream_and_device():
    from zero_sharded_mixed_flatparameter_gb300 import _current
    from zero_sharded_mixed_flatparameter_gb300.runner import FlatStep
    assert _current.current_device() == torch.cuda.current_device()
    for stream in (torch.cuda.current_stream(), torch.cuda.Stream()):
        with torch.cuda.stream(stream):
            assert FlatStep.stream_handle() == FlatStep.stream_handle(stream) == stream.cuda_stream
            assert _current._public_stream(0) == _current.current_stream(0) == stream.cuda_stream
