"""Norm and rotation of queries and keys on the GPU against 64 bits, forward
and backward.

Tolerances.  fp32: an element is a product of a few rounded factors and one
sum of head_dim squares; with the sums' errors well below sqrt(head_dim) * 2^-24
a relative error of 2e-6 of the tensor covers it.  bf16: the 64-bit value is
rounded to bf16 as well, so that only the few elements whose fp32 value falls on
the other side of a rounding boundary differ (by 2^-7 at most): 2^-9 of the
tensor.  Gain gradients: fp32 sums of tokens * heads terms of
random sign, errors in quadrature: 5e-6 of the norm.
"""

import pytest
import torch

from muon_reference import qk64, relative, rotation_table
from zero_sharded_mixed_flatparameter_gb300 import binding as B
from zero_sharded_mixed_flatparameter_gb300 import ops

pytestmark = pytest.mark.gpu

TOL = {torch.float32: 2e-6, torch.bfloat16: 2.0 ** -9}
GAIN_TOL = 5e-6


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_sharded_mixed_flatparameter_gb300 import build_lib
    build_lib.build()
    B.load()


def inputs(tokens, hq, hk, dim, rotary, dtype, seed=0, n_positions=100, gain_dtype=torch.float32, padded=True):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.empty(shape).normal_(generator=g)

    q, k, dq, dk = (normal(tokens, h, dim).to(dtype) for h in (hq, hk, hq, hk))
    gains = [(1 + 0.1 * normal(dim)).to(gain_dtype) for _ in range(2)]
    positions = torch.randint(0, n_positions, (tokens,), generator=g, dtype=torch.int32)
    if padded and tokens > 2:
        positions[tokens // 2] = -1
        positions[tokens - 1] = n_positions
    return q, k, dq, dk, gains, rotation_table(n_positions, rotary), positions


CASES = [  # tokens, q heads, k heads, head_dim, rotary_dim
    (1, 32, 8, 64, 64), (2, 3, 1, 2, 2), (7, 4, 4, 33, 32), (5, 2, 1, 80, 32), (9, 5, 1, 96, 96),
    (33, 16, 4, 64, 64), (130, 8, 2, 128, 128), (65, 4, 1, 128, 64), (17, 3, 1, 256, 256), (31, 2, 2, 255, 128),
    (64, 1, 0, 64, 32), (64, 0, 1, 64, 32), (1000, 12, 4, 32, 32), (511, 3, 1, 72, 24), (100, 2, 1, 8, 8),
    (40, 2, 1, 24, 10), (2000, 32, 8, 64, 64)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("tokens,hq,hk,dim,rotary", CASES)
def test_forward_and_backward(tokens, hq, hk, dim, rotary, dtype, interleaved):
    q, k, dq, dk, gains, table, positions = inputs(tokens, hq, hk, dim, rotary, dtype, seed=tokens + dim)
    dev = [x.cuda() for x in (q, k, *gains, table, positions)]
    out = ops.qk_norm_rope(*dev, interleaved=interleaved)
    back = ops.qk_norm_rope_backward(dq.cuda(), dk.cuda(), *dev, interleaved=interleaved)
    for i, (x, dy, gain) in enumerate(((q, dq, gains[0]), (k, dk, gains[1]))):
        x64, g64 = x.double().requires_grad_(), gain.double().requires_grad_()
        want = qk64(x64, g64, table, positions, 1e-6, interleaved)
        assert out[i].shape == x.shape and out[i].dtype == dtype
        assert relative(out[i], want.detach().to(dtype)) <= TOL[dtype]
        dead = (positions < 0) | (positions >= 100)
        assert (out[i].cpu()[dead] == 0).all() and (back[i].cpu()[dead] == 0).all()
        if x.numel() == 0:
            assert (back[2 + i] == 0).all()
            continue
        dx, dgain = torch.autograd.grad(want, (x64, g64), dy.double())
        scale = max(float(dx.norm()), 1e-3 * float(dy.double().norm()))
        assert float((back[i].cpu().double() - dx.to(dtype).double()).norm()) <= TOL[dtype] * scale
        assert relative(back[2 + i], dgain) <= GAIN_TOL


def test_gradients_against_differences():
    tokens, hq, hk, dim, rotary = 40, 4, 2, 64, 48
    q, k, dq, dk, gains, table, positions = inputs(tokens, hq, hk, dim, rotary, torch.float32, 5)
    g = torch.Generator().manual_seed(6)
    args = [x.cuda() for x in (q, k, *gains)]
    rest = [table.cuda(), positions.cuda()]
    grads = ops.qk_norm_rope_backward(dq.cuda(), dk.cuda(), *args, *rest)
    for i in range(4):
        direction = torch.empty(args[i].shape).normal_(generator=g).cuda()
        step = 1e-2
        value = []
        for sign in (1, -1):
            moved = list(args)
            moved[i] = args[i] + sign * step * direction
            oq, ok = ops.qk_norm_rope(*moved, *rest)
            value.append(float((oq.double() * dq.cuda()).sum() + (ok.double() * dk.cuda()).sum()))
        slope = (value[0] - value[1]) / (2 * step)
        want = float((grads[i].double() * direction).sum())
        # third-order term of a central difference (step^2) and fp32 outputs, both against the gradient's size
        size = float(grads[i].double().norm())
        assert abs(slope - want) <= 2e-3 * size, i


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_strided_and_in_place(dtype):
    tokens, hq, hk, dim = 50, 6, 2, 64
    q, k, dq, dk, gains, table, positions = inputs(tokens, hq, hk, dim, 64, dtype, 7)
    rest = [x.cuda() for x in (*gains, table, positions)]
    want = ops.qk_norm_rope(q.cuda(), k.cuda(), *rest)
    want_back = ops.qk_norm_rope_backward(dq.cuda(), dk.cuda(), q.cuda(), k.cuda(), *rest)
    for pad in (0, 1, 8):  # one projection's output, at several alignments; heads before tokens
        fused = torch.full((tokens, (hq + hk) * dim + pad), float("nan"), dtype=dtype, device="cuda")
        fq = fused[:, :hq * dim].unflatten(1, (hq, dim))
        fk = fused[:, hq * dim:(hq + hk) * dim].unflatten(1, (hk, dim))
        fq.copy_(q)
        fk.copy_(k)
        ops.qk_norm_rope(fq, fk, *rest, out=(fq, fk))
        assert torch.equal(fq, want[0]) and torch.equal(fk, want[1]), pad
        assert fused[:, (hq + hk) * dim:].isnan().all()
    hq_first = q.cuda().transpose(0, 1).contiguous().transpose(0, 1)
    got = ops.qk_norm_rope(hq_first, k.cuda(), *rest)
    assert torch.equal(got[0], want[0])
    a, b = dq.cuda(), dk.cuda()
    got = ops.qk_norm_rope_backward(a, b, hq_first, k.cuda(), *rest, out=(a, b))
    assert got[0] is a
    for x, y in zip(got, want_back):
        assert torch.equal(x, y)


def test_no_gain_no_rotation_no_positions():
    q, k, dq, dk, _, _, _ = inputs(20, 3, 1, 64, 0, torch.float32, 8)
    empty = torch.empty((20, 0))
    out = ops.qk_norm_rope(q.cuda(), k.cuda(), None, None, empty.cuda())
    assert relative(out[0], qk64(q.double(), None, empty, torch.arange(20), 1e-6, False)) <= 2e-6
    table = rotation_table(20, 64)
    out = ops.qk_norm_rope(q.cuda(), k.cuda(), None, None, table.cuda())
    assert relative(out[1], qk64(k.double(), None, table, torch.arange(20), 1e-6, False)) <= 2e-6
    back = ops.qk_norm_rope_backward(dq.cuda(), dk.cuda(), q.cuda(), k.cuda(), None, None, table.cuda())
    x = q.double().requires_grad_()
    dx, = torch.autograd.grad(qk64(x, None, table, torch.arange(20), 1e-6, False), x, dq.double())
    assert relative(back[0], dx) <= 2e-6


@pytest.mark.parametrize("gain_dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_gains_and_their_gradient_in_the_flat_buffers(gain_dtype):
    # gains read from, and gradients written to, odd offsets of flat buffers
    q, k, dq, dk, gains, table, positions = inputs(77, 4, 2, 64, 64, torch.bfloat16, 9, gain_dtype=gain_dtype)
    flat = torch.full((300,), 7.0, dtype=gain_dtype, device="cuda")
    grad = torch.full((300,), 7.0, dtype=gain_dtype, device="cuda")
    gq, gk = flat[3:67], flat[101:165]
    gq.copy_(gains[0])
    gk.copy_(gains[1])
    rest = [x.cuda() for x in (table, positions)]
    back = ops.qk_norm_rope_backward(dq.cuda(), dk.cuda(), q.cuda(), k.cuda(), gq, gk, *rest,
                                     gain_out=(grad[3:67], grad[101:165]))
    want = ops.qk_norm_rope_backward(dq.cuda(), dk.cuda(), q.cuda(), k.cuda(), gains[0].cuda(), gains[1].cuda(), *rest)
    assert torch.equal(back[0], want[0]) and torch.equal(back[1], want[1])
    assert torch.equal(back[2], want[2].to(gain_dtype)) and torch.equal(back[3], want[3].to(gain_dtype))
    keep = torch.ones(300, dtype=torch.bool)
    keep[3:67] = keep[101:165] = False
    assert (grad.cpu()[keep] == 7.0).all()


def test_all_padding_and_no_tokens():
    q, k, dq, dk, gains, table, positions = inputs(12, 2, 1, 64, 64, torch.bfloat16, 10)
    positions[:] = -1
    q[3] = float("nan")
    dq[4] = float("inf")
    dev = [x.cuda() for x in (q, k, *gains, table, positions)]
    assert (ops.qk_norm_rope(*dev)[0] == 0).all()
    for x in ops.qk_norm_rope_backward(dq.cuda(), dk.cuda(), *dev):
        assert (x == 0).all(), "what is behind padding reaches no sum"
    none = [x[:0].contiguous() for x in (dev[0], dev[1])]
    out = ops.qk_norm_rope(*none, *dev[2:5], positions[:0].cuda())
    assert out[0].shape == (0, 2, 64)
    back = ops.qk_norm_rope_backward(*none, *none, *dev[2:5], positions[:0].cuda())
    assert (back[2] == 0).all() and (back[3] == 0).all()


@pytest.mark.parametrize("dim,rotary", [(64, 64), (72, 24), (80, 32)])
def test_no_eps(dim, rotary):
    # with eps 0 nothing that is not a real head (padding, lanes without one) may reach a sum
    q, k, dq, dk, gains, table, positions = inputs(37, 5, 3, dim, rotary, torch.float32, 15)
    dev = [x.cuda() for x in (q, k, *gains, table, positions)]
    out = ops.qk_norm_rope(*dev, eps=0.0)
    back = ops.qk_norm_rope_backward(dq.cuda(), dk.cuda(), *dev, eps=0.0)
    x, gain = k.double().requires_grad_(), gains[1].double().requires_grad_()
    want = qk64(x, gain, table, positions, 0.0, False)
    assert relative(out[1], want.detach()) <= 2e-6
    dx, dgain = torch.autograd.grad(want, (x, gain), dk.double())
    assert relative(back[1], dx) <= 2e-6 and relative(back[3], dgain) <= GAIN_TOL


def test_zero_rows_and_large_values():
    q, k, dq, dk, gains, table, positions = inputs(6, 2, 1, 64, 64, torch.float32, 11, padded=False)
    q[0] = 0
    q[1] *= 1e15
    q[2] *= 1e-15
    dev = [x.cuda() for x in (q, k, *gains, table, positions)]
    out = ops.qk_norm_rope(*dev)[0].cpu()
    want = qk64(q.double(), gains[0].double(), table, positions, 1e-6, False)
    assert (out[0] == 0).all()
    for t in range(6):
        assert relative(out[t], want[t]) <= 2e-6
    back = ops.qk_norm_rope_backward(dq.cuda(), dk.cuda(), *dev)[0].cpu()
    x = q.double().requires_grad_()
    dx, = torch.autograd.grad(qk64(x, gains[0].double(), table, positions, 1e-6, False), x, dq.double())
    for t in range(6):
        assert relative(back[t], dx[t]) <= 2e-6 if t != 1 else back[t].isfinite().all()


def test_reproducible_streams_and_capture():
    q, k, dq, dk, gains, table, positions = inputs(3000, 8, 2, 64, 64, torch.bfloat16, 12)
    dev = [x.cuda() for x in (q, k, *gains, table, positions)]
    d = (dq.cuda(), dk.cuda())
    want = ops.qk_norm_rope_backward(*d, *dev)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = ops.qk_norm_rope_backward(*d, *dev)
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(want, other):
        assert torch.equal(a, b)
    out = tuple(torch.empty_like(x) for x in dev[:2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.qk_norm_rope(*dev, out=out)
    graph.replay()
    for a, b in zip(out, ops.qk_norm_rope(*dev)):
        assert torch.equal(a, b)


def test_long_sequence_offsets():
    # token offsets past 2^31 elements: the last tokens of a long strided buffer
    tokens, dim = 40, 64
    stride = (1 << 31) // (tokens - 2) // 64 * 64 + 64
    big = torch.empty((tokens - 1) * stride + dim, dtype=torch.bfloat16, device="cuda")
    q = big.as_strided((tokens, 1, dim), (stride, dim, 1))
    src, _, _, _, gains, table, positions = inputs(tokens, 1, 1, dim, 64, torch.bfloat16, 13, padded=False)
    q.copy_(src)
    rest = [x.cuda() for x in (*gains, table, positions)]
    k = src.cuda()
    out = ops.qk_norm_rope(q, k, *rest, out=(q, torch.empty_like(k)))
    assert torch.equal(out[0].contiguous(), ops.qk_norm_rope(k, k, rest[0], rest[0], *rest[2:])[0])


def test_autograd():
    q, k, dq, dk, gains, table, positions = inputs(30, 3, 1, 64, 32, torch.float32, 14)
    leaves = [x.cuda().requires_grad_() for x in (q, k, *gains)]
    out = ops.qk_norm_rope_autograd(*leaves, table.cuda(), positions.cuda())
    torch.autograd.backward(out, (dq.cuda(), dk.cuda()))
    want = ops.qk_norm_rope_backward(dq.cuda(), dk.cuda(), *[x.detach() for x in leaves], table.cuda(), positions.cuda())
    for leaf, w in zip(leaves, want):
        assert torch.equal(leaf.grad, w)


def config(**over):
    base = dict(q_heads=2, k_heads=1, head_dim=64, rotary_dim=64, interleaved=0, dtype=1, gain_dtype=1, eps=1e-6,
                n_positions=16)
    base.update(over)
    return B.zero_qk_config(*base.values())


@pytest.mark.parametrize("over", [
    dict(q_heads=-1), dict(head_dim=0), dict(head_dim=1, rotary_dim=0), dict(head_dim=257), dict(rotary_dim=3), dict(rotary_dim=66),
    dict(rotary_dim=-2), dict(interleaved=2), dict(dtype=2), dict(gain_dtype=-1), dict(eps=-1.0),
    dict(eps=float("nan")), dict(n_positions=-1), dict(tokens=-1), dict(q=0), dict(k=0), dict(q_out=0), dict(table=0),
    dict(q=2), dict(positions=2), dict(q_gain=2), dict(stride=-1), dict(workspace=0), dict(workspace_bytes=1),
    dict(dgain_dtype=5), dict(dq=0),
], ids=str)
def test_refusals(over):
    x = torch.zeros(1 << 16, device="cuda")
    p = x.data_ptr()

    def run(**o):
        cfg = config(**{k: v for k, v in o.items() if k in dict(B.zero_qk_config._fields_)})
        tokens = o.get("tokens", 4)

        def at(name, default):  # 0: NULL, 2: misaligned
            v = o.get(name)
            return default if v is None else (0 if v == 0 else default + v)

        stride = o.get("stride", 128)
        q, k = B.zero_heads(at("q", p), stride, 64), B.zero_heads(at("k", p), 64, 64)
        qo, ko = B.zero_heads(at("q_out", p + 65536), 128, 64), B.zero_heads(p + 131072, 64, 64)
        back = {"workspace", "workspace_bytes", "dgain_dtype", "dq"} & set(o)
        if not back:
            B.zero_qk_norm_rope(cfg, tokens, q, k, at("q_gain", p), p, at("table", p), at("positions", p + 8192), qo, ko)
        else:
            dq = B.zero_heads(at("dq", p), 128, 64)
            ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
            B.zero_qk_norm_rope_backward(cfg, tokens, dq, k, q, k, p, p, p, p + 8192, qo, ko, p + 200000, p + 204000,
                                         o.get("dgain_dtype", 1), at("workspace", ws.data_ptr()),
                                         o.get("workspace_bytes", 1 << 20))
        torch.cuda.synchronize()

    run()
    with pytest.raises(B.ZeroError) as e:
        run(**over)
    assert e.value.status == B.ZERO_EINVAL


def test_tensor_checks():
    q, k, dq, dk, gains, table, positions = [x if isinstance(x, list) else x.cuda()
                                             for x in inputs(4, 2, 1, 64, 64, torch.float32)]
    g = [x.cuda() for x in gains]
    good = [q, k, *g, table, positions]
    ops.qk_norm_rope(*good)
    for i, bad in ((0, q.half()), (0, q.transpose(1, 2)), (0, q[0]), (1, k[:3]), (1, k.bfloat16()), (2, g[0][:5]),
                   (3, g[1].bfloat16()), (4, table.double()), (4, table[0]), (5, positions.long()), (5, positions[:2]),
                   (5, positions.cpu())):
        args = list(good)
        args[i] = bad
        with pytest.raises(ValueError):
            ops.qk_norm_rope(*args)
    with pytest.raises(ValueError):
        ops.qk_norm_rope_backward(dk, dk, *good)
