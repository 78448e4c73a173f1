"""Checks of the operators that need no device (not gpu)."""

import random

import pytest
import torch

from zero_sharded_mixed_flatparameter_gb300 import ops


def elements(x):
    """The byte addresses of a tensor's elements."""
    at = torch.zeros(x.shape, dtype=torch.int64)
    for d, (n, stride) in enumerate(zip(x.shape, x.stride())):
        at += (torch.arange(n) * stride).view([-1 if e == d else 1 for e in range(x.dim())])
    return [x.data_ptr() + a * x.element_size() for a in at.flatten().tolist()]


def refused(outs, ins):
    try:
        ops._check_memory(outs, ins)
        return False
    except ValueError:
        return True


def random_view(rng, buffer):
    shape = [rng.randint(1, 5) for _ in range(3)]
    strides = [rng.choice([0, 1, 2, 4, 5, 6, 8, 20, 24, 40]) for _ in range(2)] + [1]
    rng.shuffle(shape)
    reach = sum((n - 1) * s for n, s in zip(shape, strides))
    return buffer.as_strided(shape, strides, rng.randint(0, buffer.numel() - 1 - reach))


def test_every_overlap_is_found():
    # against the sets of addresses; what cannot be told apart may be refused, too
    rng, buffer, allowed = random.Random(5), torch.empty(512), 0
    for _ in range(4000):
        out, other = random_view(rng, buffer), random_view(rng, buffer)
        mine, theirs = elements(out), elements(other)
        if not refused((out,), ((), (other,))):
            allowed += 1
            assert len(set(mine)) == len(mine) and not set(mine) & set(theirs), (out.stride(), other.stride())
    assert allowed > 400


@pytest.mark.parametrize("tokens", [1, 7])
def test_usual_layouts_are_allowed(tokens):
    fused = torch.empty(tokens, 8 * 64 + 3)
    q, k = fused[:, :4 * 64].unflatten(1, (4, 64)), fused[:, 4 * 64:6 * 64].unflatten(1, (2, 64))
    v = fused[:, 6 * 64:8 * 64].unflatten(1, (2, 64))
    ops._check_memory((q, k), ((q,), (k,)))                              # in place
    ops._check_memory((torch.empty(tokens, 4, 64), v), ((q,), (k,)))     # beside them in one buffer
    heads_first = torch.empty(4, tokens, 64).transpose(0, 1)
    ops._check_memory((heads_first, k), ((q, heads_first), (k,)))
    grouped = torch.empty(tokens, 2, 3, 64)                              # two queries and a key per group
    ops._check_memory((grouped[:, :, 0], grouped[:, :, 2]), ((grouped[:, :, 0],), (grouped[:, :, 2],)))
    halves = torch.empty(2, 5, 40)
    ops._check_memory((halves[:, :, :16],), ((), (halves[:, :, 16:32],)))
    ops._check_memory((torch.empty(0, 4, 64), torch.empty(0, 2, 64)), ((q,), (k,)))


def test_overlaps_are_refused():
    x = torch.empty(6, 4, 64)
    other = torch.empty(6, 4, 64)
    assert refused((x,), ((), (x,)))                                     # an output that may be no input
    assert refused((x, x), ((other,), (other,)))                         # twice the same
    assert refused((x[1:],), ((x[:-1],),))                               # shifted by a token
    assert refused((other, x), ((x,), (other,)))                         # crossed
    assert refused((other[:1].expand(6, 4, 64),), ((x,),))               # one row for all
    assert refused((x.transpose(0, 1)[:, :4],), ((x[:4],),))             # the same memory in another order
    vector = torch.empty(10)
    assert refused((vector[:6], vector[4:]), ()) and not refused((vector[:5], vector[5:]), ())
