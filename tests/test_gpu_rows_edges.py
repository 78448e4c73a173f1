"""Calls of the layer norm, the 8-bit form and the embedding that the documentation
allows at its edges: nothing to do inside a captured graph, inputs without rows
or leading dimensions through autograd, several threads and graphs at once."""

import threading

import pytest
import torch

from rows_reference import E4M3, INT8
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


def test_no_rows_behind_a_copy_in_a_graph():
    # the join of no rows follows whatever stands before it in the stream: a copy, nothing, a fill
    x, w, stats = torch.empty(0, 40, device="cuda"), normal(40), torch.empty(0, 2, device="cuda")
    source, target = normal(1 << 20), torch.zeros(1 << 20, device="cuda")
    dw, db = torch.full((40,), 7.0, device="cuda"), torch.full((40,), 7.0, device="cuda")
    for before in (lambda: target.copy_(source), lambda: None, lambda: target.zero_()):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            before()
            ops.layer_norm_backward(x, x, w, stats, weight_out=dw, bias_out=db)
            again = ops.embedding_backward(x, torch.empty(0, dtype=torch.int64, device="cuda"), 5)
        for _ in range(2):
            dw.fill_(7.0)
            db.fill_(7.0)
            graph.replay()
            assert (dw == 0).all() and (db == 0).all() and (again == 0).all()


@pytest.mark.parametrize("pack", [None, E4M3, INT8], ids=["whole", "e4m3", "int8"])
@pytest.mark.parametrize("shape", [(0, 40), (3, 0, 40), (40,), (1, 40), (2, 1, 3, 40)], ids=str)
def test_shapes_through_autograd(shape, pack):
    x, w, b = normal(*shape).requires_grad_(), normal(40, seed=1).requires_grad_(), normal(40, seed=2).requires_grad_()
    dy = normal(*shape, seed=3)
    y = ops.layer_norm_autograd(x, w, b, pack=pack)
    y.backward(dy)
    assert y.shape == x.grad.shape == x.shape
    plain = [t.detach().reshape(-1, 40) if t is x else t.detach() for t in (x, w, b)]
    want, stats, *packed = ops.layer_norm(*plain, pack=pack)
    grads = ops.layer_norm_backward(dy.reshape(-1, 40), packed[0] if packed else plain[0], plain[1], stats)
    assert torch.equal(y.reshape(-1, 40), want)
    for got, g in zip((x.grad.reshape(-1, 40), w.grad, b.grad), grads):
        assert torch.equal(got, g)
    ids = torch.zeros(shape[:-1], dtype=torch.int64, device="cuda")
    table = normal(4, 40, seed=4).requires_grad_()
    out = ops.embedding_autograd(ids, table)
    assert out.shape == shape
    out.backward(dy)
    assert torch.equal(table.grad, ops.embedding_backward(dy, ids, 4))


def run(x, dy, w, ids, form):
    y, stats, packed = ops.layer_norm(x, w, pack=form)
    return (y, *ops.layer_norm_backward(dy, packed, w, stats), *ops.layer_norm_backward(dy, x, w, stats),
            ops.unpack_activations(packed), ops.embedding_backward(dy, ids, 50), ops.embedding(ids, x[:50]))


def test_threads_with_streams_of_their_own():
    sizes, wrong = [(700, 1000), (701, 999), (5000, 64), (300, 8200)], []
    args = [(normal(r, c), normal(r, c, seed=1), normal(c), torch.arange(r, device="cuda") % 60 - 3, form)
            for (r, c), form in zip(sizes, (E4M3, INT8, INT8, E4M3))]
    wants = [run(*a) for a in args]
    torch.cuda.synchronize()

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(30):
                got = run(*args[i])
            s.synchronize()
            if not all(torch.equal(g, w) for g, w in zip(got, wants[i])):
                wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(args))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_graphs_replayed_beside_each_other():
    args = [(normal(r, c), normal(r, c, seed=1), normal(c), torch.arange(r, device="cuda") % 60 - 3, E4M3)
            for r, c in ((900, 1024), (400, 1301))]
    wants = [run(*a) for a in args]
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in args]
    for a in args:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run(*a))
        graphs.append(g)
    for out in outs:
        for t in out:
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for out, want in zip(outs, wants):
        for o, w in zip(out, want):
            assert torch.equal(o, w)
