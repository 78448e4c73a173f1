"""How long the Muon step's workspace lives: repeated configurations, captured
steps, other streams."""

import gc

import pytest
import torch

from gpu_common import ensure_built
from test_gpu_muon import LR, MU, WD, grads_for, make, mlp, step

pytestmark = pytest.mark.gpu

NAMES = ("master", "exp_avg", "exp_avg_sq", "param16")


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def equal(a, b):
    return all(torch.equal(getattr(a, n), getattr(b, n)) for n in NAMES)


def taken(nbytes):
    """Tensors over whatever the allocator has to give of that size, filled."""
    gc.collect()
    return [torch.full((nbytes // 4,), 7.0, device="cuda") for _ in range(4)]


def test_momentum_warm_up_allocates_nothing():
    pl, shapes = mlp([150, 300, 140])
    fs = make(pl, shapes, 2)
    before = torch.cuda.memory_allocated()
    for t in range(5):
        fs.enable_muon(shapes, lr=LR, momentum=0.8 + 0.03 * t, weight_decay=WD)
        assert torch.cuda.memory_allocated() == before
        step(fs, grads_for(fs, pl, 2, "bf16", t + 1))
    fs.disable_muon()
    fs.enable_muon(shapes, lr=LR)
    assert torch.cuda.memory_allocated() == before


def test_a_smaller_configuration_uses_the_same_workspace():
    pl, shapes = mlp([150, 300, 140])
    fs, fresh = make(pl, shapes, 2), make(pl, [shapes[0], None, None, None], 2)
    fs.enable_muon([shapes[0], None, None, None], lr=LR, momentum=MU, weight_decay=WD)
    grads = grads_for(fs, pl, 2, "bf16", 1)
    step(fs, grads)
    step(fresh, grads)
    assert equal(fs, fresh)


@pytest.mark.parametrize("then", ["larger", "disable"])
def test_captured_steps_keep_their_workspace(then):
    pl, shapes = mlp([150, 300, 140])
    first = [shapes[0], None, None, None]
    eager, fs = make(pl, first, 2), make(pl, first, 2)
    nbytes = fs._muon_ws[-1].numel()
    fs.enable_capturable(8)
    static = [torch.empty(fs.padded, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for s, g in zip(static, grads_for(fs, pl, 2, "bf16", 1)):
        s.copy_(g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(fs, static)
    if then == "larger":
        fs.enable_muon(shapes, lr=LR, momentum=0.5)
    else:
        fs.disable_muon()
    others = taken(nbytes)
    for t in range(3):
        grads = grads_for(fs, pl, 2, "bf16", t + 1)
        for s, g in zip(static, grads):
            s.copy_(g)
        graph.replay()
        step(eager, grads)
        assert equal(fs, eager), t
    assert all((x == 7.0).all() for x in others), "memory of other tensors is left alone"


def test_step_in_flight_on_another_stream():
    pl, shapes = mlp([500, 1500, 700])
    first = [shapes[0], None, None, None]
    fs, eager = make(pl, first, 2), make(pl, first, 2)
    grads = grads_for(fs, pl, 2, "bf16", 1)
    step(eager, grads)
    nbytes = fs._muon_ws[-1].numel()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    fs.reduce_grads(-1, grads, stream=side)
    fs.step(stream=side)
    fs.post_step(stream=side)
    fs.enable_muon(shapes, lr=LR)
    others = taken(nbytes)
    torch.cuda.synchronize()
    assert equal(fs, eager)
    assert all((x == 7.0).all() for x in others)
