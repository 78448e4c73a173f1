"""Trains one attention block with data-parallel replicas: norm and rotation of
queries and keys in one pass (forward and backward), the replicas' gradients in
flat buffers, and one optimizer step in which the four projections take the
orthogonalised (Muon) update and the two gains stay with AdamW.

The block learns to reproduce another block of random weights.  Run from the
repository's root on a GPU:  python examples/train_muon.py [steps]
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from zero_sharded_mixed_flatparameter_gb300 import ops  # noqa: E402
from zero_sharded_mixed_flatparameter_gb300.runner import FlatStep  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM, SEQUENCE = 256, 4, 2, 64, 128
SHAPES = [(HEADS * DIM, HIDDEN), (KV_HEADS * DIM, HIDDEN), (KV_HEADS * DIM, HIDDEN), (HIDDEN, HEADS * DIM)]


def rotation_table(positions: int) -> torch.Tensor:
    freq = 10000.0 ** (-torch.arange(DIM // 2, device="cuda", dtype=torch.float64) / (DIM // 2))
    angle = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def block(x, weights, table, positions):
    """x: (sequences * SEQUENCE, HIDDEN); weights: q, k, v, o projections and the two gains, bf16."""
    wq, wk, wv, wo, q_gain, k_gain = weights
    q = (x @ wq.T).view(-1, HEADS, DIM)
    k = (x @ wk.T).view(-1, KV_HEADS, DIM)
    v = (x @ wv.T).view(-1, SEQUENCE, KV_HEADS, DIM)
    q, k = ops.qk_norm_rope_autograd(q, k, q_gain, k_gain, table, positions)
    q, k = q.view(-1, SEQUENCE, HEADS, DIM), k.view(-1, SEQUENCE, KV_HEADS, DIM)
    k, v = (t.repeat_interleave(HEADS // KV_HEADS, dim=2) for t in (k, v))
    score = torch.einsum("bqhd,bkhd->bhqk", q, k).float() / DIM ** 0.5
    future = torch.ones(SEQUENCE, SEQUENCE, dtype=torch.bool, device="cuda").triu(1)
    weight = score.masked_fill(future, float("-inf")).softmax(-1).to(v.dtype)
    return torch.einsum("bhqk,bkhd->bqhd", weight, v).reshape(-1, HEADS * DIM) @ wo.T


def train(steps: int = 60, replicas: int = 2, sequences: int = 4, seed: int = 0):
    """Returns the mean loss (relative to the target's variance) of every step."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.empty(shape, device="cuda").normal_(0.0, std, generator=gen)

    teacher = [normal(*s, std=HIDDEN ** -0.5).bfloat16() for s in SHAPES] + [1 + normal(DIM, std=0.3).bfloat16()
                                                                             for _ in range(2)]
    init = [normal(*s, std=HIDDEN ** -0.5) for s in SHAPES] + [torch.ones(DIM, device="cuda") for _ in range(2)]
    numel = [p.numel() for p in init]
    fs = FlatStep(numel, [0] * len(numel), stage=2, n_ranks=replicas, lr=1e-2, adamw=True,
                  init_params=[p.reshape(-1) for p in init])
    # the projections' rate follows Adam's scale of an update; the gains' entries stay with AdamW
    fs.enable_muon([*SHAPES, None, None], lr=1e-2, weight_decay=0.0)
    table = rotation_table(SEQUENCE)
    positions = torch.arange(SEQUENCE, dtype=torch.int32, device="cuda").repeat(sequences)
    losses = []
    for _ in range(steps):
        grads, total = [], 0.0
        for _ in range(replicas):
            weights = [fs.param16[fs.param_offset(p):fs.param_offset(p) + n].view(i.shape).detach().requires_grad_()
                       for p, (n, i) in enumerate(zip(numel, init))]
            x = normal(sequences * SEQUENCE, HIDDEN).bfloat16()
            with torch.no_grad():
                target = block(x, teacher, table, positions).float()
            loss = (block(x, weights, table, positions).float() - target).square().mean() / target.square().mean()
            loss.backward()
            flat = torch.zeros(fs.padded, dtype=torch.bfloat16, device="cuda")
            for p, (n, w) in enumerate(zip(numel, weights)):
                flat[fs.param_offset(p):fs.param_offset(p) + n] = w.grad.reshape(-1)
            grads.append(flat)
            total += loss.detach()
        fs.reduce_grads(-1, grads)
        fs.step()
        fs.post_step()
        losses.append(total / replicas)
    return torch.stack(losses).tolist()


if __name__ == "__main__":
    history = train(int(sys.argv[1]) if len(sys.argv) > 1 else 60)
    for i, loss in enumerate(history):
        if i % 10 == 0 or i + 1 == len(history):
            print(f"step {i:4d}  loss {loss:.4f}")
