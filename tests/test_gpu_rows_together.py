"""The operators as a training step uses them: embedding, norms (the first one's
input kept in 8 bits), norm and rotation of queries and keys, gradients written
into a replica's flat gradient, the optimizer step over all of it."""

import math

import pytest
import torch

from muon_reference import qk64, rotation_table
from rows_reference import E4M3, INT8, pack64
from zero_sharded_mixed_flatparameter_gb300 import binding as B
from zero_sharded_mixed_flatparameter_gb300 import ops
from zero_sharded_mixed_flatparameter_gb300.runner import FlatStep

pytestmark = pytest.mark.gpu

VOCAB, HIDDEN, HEADS, DIM, SEQUENCE, SEQUENCES = 101, 64, 4, 16, 24, 3
SCALE = math.sqrt(HIDDEN)  # 8: the looked up rows are exact
TOKENS = SEQUENCE * SEQUENCES
# embedding; a layer's two projections, gains and norms; the final norm with a bias; the head
SHAPES = [(VOCAB, HIDDEN), (3 * HEADS * DIM, HIDDEN), (HIDDEN, HEADS * DIM), (DIM,), (DIM,), (HIDDEN,), (HIDDEN,),
          (HIDDEN,), (VOCAB, HIDDEN)]


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_sharded_mixed_flatparameter_gb300 import build_lib
    build_lib.build()
    B.load()


class KeptNorm64(torch.autograd.Function):
    """The RMS norm in 64 bits whose backward pass sees the rounded input."""

    @staticmethod
    def forward(ctx, x, gain, form):
        rstd = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-5)
        ctx.save_for_backward(pack64(x.float(), form)[2], rstd, gain)
        return x * rstd * gain

    @staticmethod
    def backward(ctx, dy):
        x, rstd, gain = ctx.saved_tensors
        xn, g = x * rstd, dy * gain
        return rstd * (g - xn * (g * xn).mean(-1, keepdim=True)), (dy * xn).sum(0), None


def attention(q, k, v):
    q, k, v = (t.view(SEQUENCES, SEQUENCE, HEADS, DIM) for t in (q, k, v))
    score = torch.einsum("bqhd,bkhd->bhqk", q, k) / DIM ** 0.5
    future = torch.ones(SEQUENCE, SEQUENCE, dtype=torch.bool, device=q.device).triu(1)
    return torch.einsum("bhqk,bkhd->bqhd", score.masked_fill(future, float("-inf")).softmax(-1), v).reshape(TOKENS, -1)


def loss_of(logits, targets):
    return (logits.logsumexp(-1) - logits.gather(1, targets[:, None])[:, 0]).mean()


def step(weights, ids, targets, table, positions, pack):
    """The framework's operators, recording their gradients."""
    emb, wqkv, wo, qg, kg, gain, final, bias, head = weights
    x = ops.embedding_autograd(ids, emb, scale=SCALE)
    h = ops.layer_norm_autograd(x, gain, center=False, pack=pack)
    q, k, v = (h @ wqkv.T).view(TOKENS, 3, HEADS, DIM).unbind(1)
    q, k = ops.qk_norm_rope_autograd(q, k, qg, kg, table, positions)
    x = x + attention(q, k, v) @ wo.T
    return loss_of(ops.layer_norm_autograd(x, final, bias) @ head.T, targets)


def step64(weights, ids, targets, table, positions, pack):
    emb, wqkv, wo, qg, kg, gain, final, bias, head = weights
    x = SCALE * emb[ids.clamp(min=0)] * (ids >= 0)[:, None]
    h = KeptNorm64.apply(x, gain, pack) if pack is not None else x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-5) * gain
    q, k, v = (h @ wqkv.T).view(TOKENS, 3, HEADS, DIM).unbind(1)
    q, k = (qk64(t, g, table, positions, 1e-6, False) for t, g in ((q, qg), (k, kg)))
    x = x + attention(q, k, v) @ wo.T
    d = x - x.mean(-1, keepdim=True)
    y = d / torch.sqrt(d.square().mean(-1, keepdim=True) + 1e-5) * final + bias
    return loss_of(y @ head.T, targets)


def inputs(seed=0):
    g = torch.Generator().manual_seed(seed)
    init = [torch.empty(s).normal_(0, 0.02 if i in (0, 8) else HIDDEN ** -0.5, generator=g) if len(s) == 2 else
            (torch.zeros(s) if i == 7 else 1 + 0.1 * torch.empty(s).normal_(generator=g)) for i, s in enumerate(SHAPES)]
    ids = torch.randint(0, VOCAB // 2, (TOKENS,), generator=g)
    ids[5] = -1
    return init, ids, torch.randint(0, VOCAB, (TOKENS,), generator=g)


@pytest.mark.parametrize("pack", [None, E4M3, INT8], ids=["whole", "e4m3", "int8"])
def test_training_step(pack):
    init, ids, targets = inputs()
    numel = [p.numel() for p in init]
    fs = FlatStep(numel, [0] * len(numel), stage=2, n_ranks=2, grad_dtype="fp32", lr=1e-2, adamw=True,
                  init_params=[p.reshape(-1).cuda() for p in init])
    fs.enable_muon([None, SHAPES[1], SHAPES[2], *[None] * 6], lr=1e-2)
    table, positions = rotation_table(SEQUENCE, DIM), torch.arange(SEQUENCE, dtype=torch.int32).repeat(SEQUENCES)
    grads = []
    for replica in range(2):
        its_ids = ids.roll(replica)
        weights = [fs.master[fs.param_offset(p):fs.param_offset(p) + n].view(s).detach().clone().requires_grad_()
                   for p, (n, s) in enumerate(zip(numel, SHAPES))]
        loss = step(weights, its_ids.cuda(), targets.cuda(), table.cuda(), positions.cuda(), pack)
        loss.backward()
        leaves = [p.double().requires_grad_() for p in init]
        want_loss = step64(leaves, its_ids, targets, table, positions, pack)
        want = torch.autograd.grad(want_loss, leaves)
        assert abs(float(loss.detach()) - float(want_loss.detach())) <= 1e-5 * float(want_loss.detach())
        flat = torch.zeros(fs.padded, device="cuda")
        for p, (w, x) in enumerate(zip(weights, want)):
            # ten operators one after another, each within 64 half steps (4e-6) of its terms, which cancel by a
            # factor of a few in the norms and the softmax: 2e-4 of the gradient's norm
            assert float((w.grad.double().cpu() - x).norm()) <= 2e-4 * float(x.norm()), p
            flat[fs.param_offset(p):fs.param_offset(p) + numel[p]] = w.grad.reshape(-1)
        assert torch.count_nonzero(weights[0].grad[VOCAB // 2:]) == 0
        grads.append(flat)
    before = fs.master.clone()
    fs.reduce_grads(-1, grads)
    fs.step()
    fs.post_step()
    moved = (fs.master != before)[:numel[0]].view(VOCAB, HIDDEN).any(1).cpu()
    used = torch.zeros(VOCAB, dtype=torch.bool)
    used[ids[ids >= 0]] = True
    assert torch.equal(moved, used), "rows without tokens keep their weights"
    fs.close()


def test_gradients_written_where_the_step_reads_them():
    """The same by hand: every gradient of a norm and of the embedding goes to the replica's flat gradient, in one
    captured graph that is replayed on other tokens."""
    init, ids, _ = inputs(1)
    numel, at = [p.numel() for p in init], 3  # an odd place in the buffer, as after other parameters
    spots = []
    for n in numel:
        spots.append(slice(at, at + n))
        at += n
    flat = torch.zeros(at + 5, dtype=torch.bfloat16, device="cuda")
    for s, p in zip(spots, init):
        flat[s] = p.reshape(-1).bfloat16().cuda()
    emb, gain, bias = flat[spots[0]].view(VOCAB, HIDDEN), flat[spots[6]], flat[spots[7]]
    dy = torch.empty(TOKENS, HIDDEN).normal_(generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    grad = torch.full_like(flat, 7.0)
    places = [grad[spots[0]].view(VOCAB, HIDDEN), grad[spots[6]], grad[spots[7]]]
    static = torch.zeros(TOKENS, dtype=torch.int64, device="cuda")

    def run(tokens, out, weight_out, bias_out):
        x = ops.embedding(tokens, emb, scale=SCALE)
        y, stats, kept = ops.layer_norm(x, gain, bias, pack=INT8)
        dx, _, _ = ops.layer_norm_backward(dy, kept, gain, stats, weight_out=weight_out, bias_out=bias_out)
        return y, ops.embedding_backward(dx, tokens, VOCAB, scale=SCALE, out=out)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, _ = run(static, *places)
    for shift in (0, 7):
        tokens = ids.roll(shift).cuda()
        static.copy_(tokens)
        graph.replay()
        fresh = [torch.empty(VOCAB, HIDDEN, dtype=torch.bfloat16, device="cuda")] + [
            torch.empty(HIDDEN, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        want = run(tokens, *fresh)
        assert torch.equal(y, want[0])
        for place, f in zip(places, fresh):
            assert torch.equal(place, f)
    untouched = torch.ones_like(flat, dtype=torch.bool)
    for p in (0, 6, 7):
        untouched[spots[p]] = False
    assert (grad[untouched] == 7.0).all()
