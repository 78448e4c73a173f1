"""Host side of the Muon step and of the operators (not gpu): configuration
checks, workspace sizes, and calls that need no device."""

import pytest

from zero_sharded_mixed_flatparameter_gb300 import binding


@pytest.fixture(scope="module")
def B():
    from zero_sharded_mixed_flatparameter_gb300 import build_lib
    build_lib.build()
    binding.load()
    return binding


@pytest.mark.parametrize("rows,cols,batch", [(1, 1, 1), (64, 64, 1), (777, 1301, 3), (8192, 2048, 4), (3, 100000, 2)])
def test_workspace_covers_what_it_holds(B, rows, cols, batch):
    need = B.zero_orthogonalize_workspace_bytes(B.make_ns_config(), rows, cols, batch)
    if min(rows, cols) <= 128 and max(rows, cols) <= 1024:
        assert need == 0  # stays in shared memory
    else:  # at the least one matrix as two fp16 halves, and a larger one's Gram matrix
        assert need >= 4 * rows * cols + (2 * min(rows, cols) ** 2 if min(rows, cols) > 128 else 0)
    assert B.zero_orthogonalize_workspace_bytes(B.make_ns_config(), rows, cols, batch + 100) >= need


@pytest.mark.parametrize("rows,cols,batch", [(0, 5, 1), (5, 0, 1), (5, 5, 0)])
def test_nothing_to_do(B, rows, cols, batch):
    assert B.zero_orthogonalize_workspace_bytes(B.make_ns_config(), rows, cols, batch) == 0
    B.zero_orthogonalize(B.make_ns_config(), rows, cols, batch, 0, 1, 5, 0, 0, 5, 0, 0, 0)


@pytest.mark.parametrize("cfg", [(0, 1.5, -0.5, 0.0, 0.0), (33, 1.5, -0.5, 0.0, 0.0), (5, float("inf"), 0.0, 0.0, 0.0),
                                 (5, 1.5, -0.5, 0.0, float("nan")), (5, 1.5, -0.5, 0.0, -1e-7),
                                 (5, 30.0, 1.0, 1.0, 0.0)])
def test_bad_iterations(B, cfg):
    with pytest.raises(B.ZeroError) as e:
        B.zero_orthogonalize_workspace_bytes(B.zero_ns_config(*cfg), 8, 8, 1)
    assert e.value.status == B.ZERO_EINVAL and B.zero_last_error(None)


@pytest.mark.parametrize("rows,cols,batch", [(-1, 2, 1), (2, -1, 1), (2, 2, -1), (1 << 31, 1, 1), (1 << 25, 1 << 25, 1)])
def test_bad_sizes(B, rows, cols, batch):
    with pytest.raises(B.ZeroError) as e:
        B.zero_orthogonalize_workspace_bytes(B.make_ns_config(), rows, cols, batch)
    assert e.value.status == B.ZERO_EINVAL


def test_plan_context(B):
    ctx = B.zero_plan(B.make_config(1, 2), [24000, 6, 24000], [0, 0, 1])
    try:
        cfg = B.make_muon_config(0.02)
        one = B.zero_muon_workspace_bytes(ctx, cfg, [160, 0, 0], [150, 0, 0])
        assert 0 < one <= B.zero_muon_workspace_bytes(ctx, cfg, [160, 0, 160], [150, 0, 150])
        assert B.zero_muon_workspace_bytes(ctx, cfg, [0, 0, 0], [0, 0, 0]) == 0
        for rows, cols in (([160, 0], [150, 0]), ([160, 0, 0], [149, 0, 0]), ([-160, 0, 0], [-150, 0, 0])):
            with pytest.raises(B.ZeroError) as e:
                B.zero_muon_workspace_bytes(ctx, cfg, rows, cols)
            assert e.value.status == B.ZERO_EINVAL
        for field, value in (("lr", float("nan")), ("momentum", 1.0), ("momentum", -0.1), ("weight_decay", -1.0),
                             ("nesterov", 2), ("scale", 5)):
            bad = B.make_muon_config(0.02)
            setattr(bad, field, value)
            with pytest.raises(B.ZeroError) as e:
                B.zero_muon_workspace_bytes(ctx, bad, [160, 0, 0], [150, 0, 0])
            assert e.value.status == B.ZERO_EINVAL
        with pytest.raises(B.ZeroError) as e:
            B.zero_enable_muon(ctx, cfg, [160, 0, 0], [150, 0, 0], 256, one)
        assert e.value.status == B.ZERO_ESTATE
        for call in (lambda: B.zero_disable_muon(ctx), lambda: B.zero_set_muon_lr(ctx, 0.1)):
            with pytest.raises(B.ZeroError) as e:
                call()
            assert e.value.status == B.ZERO_ESTATE
    finally:
        B.zero_destroy(ctx)


def test_scale_names(B):
    with pytest.raises(ValueError):
        B.make_muon_config(0.02, scale="none")
