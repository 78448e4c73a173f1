"""The Muon step of the flat buffer on the GPU: momentum bit for bit, the
update against 64 bits, everything else as without it."""

import numpy as np
import pytest
import torch

import synth_inputs as si
from gpu_common import ensure_built
from muon_reference import NS_TOL, muon_scale, orthogonalized64, relative
from zero_sharded_mixed_flatparameter_gb300 import binding as B
from zero_sharded_mixed_flatparameter_gb300.runner import FlatStep

pytestmark = pytest.mark.gpu

LR, MU, WD = 0.05, 0.95, 0.1


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def mlp(widths):
    pl = si.mlp_params(widths)
    shapes = []
    for i in range(len(widths) - 1):
        shapes += [(widths[i + 1], widths[i]), None]
    return pl, shapes


def make(pl, shapes, n=4, stage=1, dtype="bf16", seed=0, muon=True, **over):
    init = [si.normal_fp32(k, 0.02, seed + 100 + p).cuda() for p, k in enumerate(pl.numel)]
    fs = FlatStep(pl.numel, pl.unit, stage=stage, n_ranks=n, grad_dtype=dtype, lr=1e-3, weight_decay=0.1, adamw=True,
                  init_params=init)
    if muon:
        fs.enable_muon(shapes, **{**dict(lr=LR, momentum=MU, weight_decay=WD), **over})
    return fs


def grads_for(fs, pl, n, dtype, seed):
    """Replica gradients of the layout: the same real elements whatever the padding, zero pads."""
    out = []
    for r in range(n):
        g = torch.zeros(fs.padded)
        for p, k in enumerate(pl.numel):
            o = fs.param_offset(p)
            g[o:o + k] = si.normal_fp32(k, 1e-2, seed * 1009 + 31 * r + 7919 * p)
        out.append(g.to(fs.grad_dtype_torch()).cuda())
    return out


def step(fs, grads, clip=None, keep=False):
    fs.reduce_grads(-1, grads)
    if clip:
        fs.clip_grad_norm(clip, keep_reduced=keep)
    fs.step()
    fs.post_step()


def reduced(grads, coefficient=None):
    """The rank-order fp32 sum x 1/N (x the clip coefficient), every operation rounded."""
    g = grads[0].float().cpu()
    for x in grads[1:]:
        g = g + x.float().cpu()
    g = g * torch.tensor(1.0 / len(grads), dtype=torch.float32)
    return g if coefficient is None else g * coefficient


def check_matrices(fs, pl, shapes, before, g, nesterov=True, scale="rms", lr=LR, wd=WD, mu=MU):
    w0, m0 = before
    w1, m1, p16 = fs.master.cpu(), fs.exp_avg.cpu(), fs.param16.cpu()
    mu32 = torch.tensor(mu, dtype=torch.float32)
    for p, s in enumerate(shapes):
        if s is None or pl.numel[p] == 0:
            continue
        at = slice(fs.param_offset(p), fs.param_offset(p) + pl.numel[p])
        mom = mu32 * m0[at] + g[at]
        assert torch.equal(m1[at], mom), f"momentum of parameter {p}"
        u = g[at] + mu32 * mom if nesterov else mom
        o = orthogonalized64(u.view(s))
        update = (w0[at].double() * (1 - lr * wd) - w1[at].double()) / (lr * muon_scale(*s, scale))
        # the fp32 master rounds to 2^-24 of itself: an absolute error of the update
        slack = float(w0[at].abs().max()) * 2.0 ** -22 / (lr * muon_scale(*s, scale)) * np.sqrt(o.numel()) / float(o.norm())
        assert relative(update.view(s), o) <= NS_TOL + slack, f"update of parameter {p}"
        assert torch.equal(p16[at], w1[at].bfloat16()), f"param16 of parameter {p}"


def snapshot(fs):
    return fs.master.cpu().clone(), fs.exp_avg.cpu().clone()


LAYOUTS = [("toy", [32, 128, 128, 64, 64, 16], 4), ("odd", [13, 57, 131, 9], 3), ("one", [1, 1, 5], 2),
           ("wide", [300, 700, 130], 8), ("same", [96, 96, 96, 96, 96], 16)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("name,widths,n", LAYOUTS)
def test_step_against_64_bits(name, widths, n, dtype):
    pl, shapes = mlp(widths)
    fs, plain = make(pl, shapes, n, dtype=dtype), make(pl, shapes, n, dtype=dtype, muon=False)
    for t in range(3):
        grads = grads_for(fs, pl, n, dtype, t + 1)
        before = snapshot(fs)
        step(fs, grads)
        step(plain, grads)
        check_matrices(fs, pl, shapes, before, reduced(grads))
        for p, s in enumerate(shapes):  # what is not a matrix: bit for bit the Adam step
            if s is None:
                at = slice(fs.param_offset(p), fs.param_offset(p) + pl.numel[p])
                for name_ in ("master", "exp_avg", "exp_avg_sq", "param16"):
                    assert torch.equal(getattr(fs, name_)[at], getattr(plain, name_)[at]), (p, name_)
    real = torch.zeros(fs.padded, dtype=torch.bool)
    for p, k in enumerate(pl.numel):
        real[fs.param_offset(p):fs.param_offset(p) + k] = True
    for x in (fs.master, fs.exp_avg, fs.exp_avg_sq, fs.param16):
        assert (x.cpu()[~real] == 0).all(), "pads stay zero"


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("scale", ["rms", "aspect"])
def test_variants(nesterov, scale):
    pl, shapes = mlp([40, 200, 60])
    fs = make(pl, shapes, 2, nesterov=nesterov, scale=scale, weight_decay=0.0)
    for t in range(2):
        grads = grads_for(fs, pl, 2, "bf16", t + 5)
        before = snapshot(fs)
        step(fs, grads)
        check_matrices(fs, pl, shapes, before, reduced(grads), nesterov, scale, wd=0.0)


def test_stages_agree():
    # padding moves every matrix to another alignment; the results stay bit for bit
    pl, shapes = mlp([13, 57, 131, 90, 9])
    state = []
    for stage in (0, 1, 2, 3):
        fs = make(pl, shapes, 5, stage=stage)
        for t in range(2):
            step(fs, grads_for(fs, pl, 5, "bf16", t + 1))
        state.append([torch.cat([x[fs.param_offset(p):fs.param_offset(p) + k] for p, k in enumerate(pl.numel)])
                      for x in (fs.master, fs.exp_avg, fs.exp_avg_sq, fs.param16)])
    for other in state[1:]:
        for a, b in zip(state[0], other):
            assert torch.equal(a, b)


def test_unit_buffers_of_any_alignment():
    pl, shapes = mlp([13, 57, 130, 9])
    fs, whole = make(pl, shapes, 3), make(pl, shapes, 3)
    grads = grads_for(fs, pl, 3, "bf16", 4)
    step(whole, grads)
    for u in range(fs.n_units):
        _, padded, _, base = fs.layout(u)
        room = [torch.zeros(padded + 9, dtype=torch.bfloat16, device="cuda") for _ in grads]
        parts = [r[1 + i:1 + i + padded] for i, r in enumerate(room)]
        for part, g in zip(parts, grads):
            part.copy_(g[base:base + padded])
        fs.reduce_grads(u, parts)
    fs.step()
    fs.post_step()
    for name in ("master", "exp_avg", "exp_avg_sq", "param16"):
        assert torch.equal(getattr(fs, name), getattr(whole, name)), name


@pytest.mark.parametrize("keep", [False, True])
def test_clipped(keep):
    pl, shapes = mlp([24, 96, 40])
    fs = make(pl, shapes, 4)
    grads = grads_for(fs, pl, 4, "bf16", 2)
    before = snapshot(fs)
    fs.reduce_grads(-1, grads)
    fs.clip_grad_norm(0.05, keep_reduced=keep)
    fs.step()
    norm = fs.grad_norm()
    fs.post_step()
    assert norm > 0.05
    check_matrices(fs, pl, shapes, before, reduced(grads, torch.tensor(0.05 / (norm + 1e-6), dtype=torch.float64).float()))


def test_clip_kept_is_bit_identical():
    pl, shapes = mlp([24, 97, 41])
    a, b = make(pl, shapes, 4), make(pl, shapes, 4)
    for t in range(2):
        grads = grads_for(a, pl, 4, "bf16", t + 1)
        step(a, grads, clip=0.05)
        step(b, grads, clip=0.05, keep=True)
    for name in ("master", "exp_avg", "exp_avg_sq", "param16"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name


def test_captured_steps_and_their_end():
    pl, shapes = mlp([32, 128, 64])
    eager, fs = make(pl, shapes, 2), make(pl, shapes, 2)
    fs.enable_capturable(3)
    static = [torch.empty(fs.padded, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    all_grads = [grads_for(fs, pl, 2, "bf16", t + 1) for t in range(4)]
    for s, g in zip(static, all_grads[0]):
        s.copy_(g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(fs, static)
    for t in range(4):
        for s, g in zip(static, all_grads[t]):
            s.copy_(g)
        graph.replay()
        if t < 3:
            step(eager, all_grads[t])
        # the fourth replay is past the table: it must change nothing
        for name in ("master", "exp_avg", "exp_avg_sq", "param16"):
            assert torch.equal(getattr(fs, name), getattr(eager, name)), (t, name)
    fs.disable_capturable()


def test_nonfinite_count_and_zero_gradients():
    pl, shapes = mlp([16, 48, 16])
    fs = make(pl, shapes, 2)
    counter = torch.zeros(1, dtype=torch.int64, device="cuda")
    fs.count_nonfinite(counter)
    zero = [torch.zeros(fs.padded, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    before = snapshot(fs)
    step(fs, zero)
    assert counter.item() == 0
    at = slice(0, pl.numel[0])
    decay = torch.tensor(1 - np.float64(np.float32(LR)) * np.float64(np.float32(WD)), dtype=torch.float64).float()
    assert torch.equal(fs.master.cpu()[at], before[0][at] * decay), "no gradient, no momentum: decay alone"
    zero[0][3] = float("nan")
    zero[1][16 * 48 + 2] = float("inf")
    step(fs, zero)
    assert counter.item() == 2


def test_checkpoint_resumes():
    pl, shapes = mlp([20, 70, 33])
    a = make(pl, shapes, 4, stage=1)
    for t in range(2):
        step(a, grads_for(a, pl, 4, "bf16", 1))
    saved, t = a.export_state()
    b = make(pl, shapes, 2, stage=3, seed=50)
    b.import_state(*saved, t)
    ga = grads_for(a, pl, 1, "bf16", 9)
    step(a, ga * 4)
    gb = grads_for(b, pl, 1, "bf16", 9)
    step(b, gb * 2)  # identical replicas: the same average at any N
    for (xa, xb) in zip(a.export_state()[0], b.export_state()[0]):
        assert torch.equal(xa, xb)


def test_many_units_and_more_matrices_than_one_launch():
    widths = [12] * 72
    pl, shapes = mlp(widths)
    fs = make(pl, shapes, 2)
    grads = grads_for(fs, pl, 2, "bf16", 3)
    before = snapshot(fs)
    step(fs, grads)
    check_matrices(fs, pl, shapes, before, reduced(grads))


def test_enable_disable_and_rates():
    pl, shapes = mlp([16, 40, 8])
    fs, adam = make(pl, shapes, 2), make(pl, shapes, 2, muon=False)
    fs.disable_muon()
    grads = grads_for(fs, pl, 2, "bf16", 1)
    step(fs, grads)
    step(adam, grads)
    assert torch.equal(fs.master, adam.master)
    fs.enable_muon(shapes, lr=LR)
    fs.set_muon_lr(0.0)
    before = fs.master.clone()
    step(fs, grads)
    at = slice(0, pl.numel[0])
    assert torch.equal(fs.master[at], before[at])
    with pytest.raises(B.ZeroError) as e:
        fs.set_muon_lr(float("nan"))
    assert e.value.status == B.ZERO_EINVAL
    fs.disable_muon()
    for call in (fs.disable_muon, lambda: fs.set_muon_lr(0.1)):
        with pytest.raises(B.ZeroError) as e:
            call()
        assert e.value.status == B.ZERO_ESTATE


@pytest.mark.parametrize("over,status", [
    (dict(shapes=[(40, 16)]), B.ZERO_EINVAL), (dict(shapes=[(16, 39), None, (8, 40), None]), B.ZERO_EINVAL),
    (dict(shapes=[(-16, -40), None, (8, 40), None]), B.ZERO_EINVAL), (dict(lr=float("inf")), B.ZERO_EINVAL),
    (dict(momentum=1.0), B.ZERO_EINVAL), (dict(weight_decay=-0.1), B.ZERO_EINVAL), (dict(steps=0), B.ZERO_EINVAL),
    (dict(coefficients=(30.0, 1.0, 1.0)), B.ZERO_EINVAL),
], ids=str)
def test_refusals(over, status):
    pl, shapes = mlp([16, 40, 8])
    fs = make(pl, shapes, 2, muon=False)
    args = {**dict(shapes=shapes, lr=LR), **over}
    with pytest.raises(B.ZeroError) as e:
        fs.enable_muon(args.pop("shapes"), **args)
    assert e.value.status == status
    grads = grads_for(fs, pl, 2, "bf16", 1)
    step(fs, grads)  # the context is as it was


def test_state_refusals():
    pl, shapes = mlp([140, 300, 8])
    fs = make(pl, shapes, 2, muon=False)
    fs.reduce_grads(-1, grads_for(fs, pl, 2, "bf16", 1))
    fs.step()
    with pytest.raises(B.ZeroError) as e:
        fs.enable_muon(shapes, lr=LR)
    assert e.value.status == B.ZERO_ESTATE
    fs.post_step()
    fs.enable_muon(shapes, lr=LR)
    cfg = B.make_muon_config(LR)
    rows, cols = [s[0] if s else 0 for s in shapes], [s[1] if s else 0 for s in shapes]
    need = B.zero_muon_workspace_bytes(fs.ctx, cfg, rows, cols)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    host = torch.empty(need + 256, dtype=torch.uint8)
    for ptr, size in ((0, need), (ws.data_ptr(), need - 1), (ws.data_ptr() + 16, need),
                      ((host.data_ptr() + 255) // 256 * 256, need)):
        with pytest.raises(B.ZeroError) as e:
            B.zero_enable_muon(fs.ctx, cfg, rows, cols, ptr, size)
        assert e.value.status == B.ZERO_EINVAL
    init = [torch.zeros(k, device="cuda") for k in pl.numel]
    off = FlatStep(pl.numel, pl.unit, stage=2, n_ranks=2, init_params=init, offload=True)
    with pytest.raises(B.ZeroError) as e:
        off.enable_muon(shapes, lr=LR)
    assert e.value.status == B.ZERO_ENOTSUP


def test_llama_layer_shapes():
    # one decoder layer of the hidden-1024 model: wide, tall and square matrices
    h, inter, kv = 1024, 2048, 256
    pl = si.llama_params(h, inter, 16, 4, 1, 0, embed=False, head=False, final_norm=False)
    shapes = [(h, h), (kv, h), (kv, h), (h, h), (inter, h), (inter, h), (h, inter), None, None]
    fs = make(pl, shapes, 8)
    grads = grads_for(fs, pl, 8, "bf16", 1)
    before, timeouts = snapshot(fs), fs.kernel_timeouts()
    step(fs, grads)
    check_matrices(fs, pl, shapes, before, reduced(grads))
    assert fs.kernel_timeouts() == timeouts


def test_nothing_outside_the_buffers_is_written():
    for widths in ([13, 57, 131, 9], [260, 300, 140], [30, 2000]):
        pl, shapes = mlp(widths)
        init = [si.normal_fp32(k, 0.02, 100 + p).cuda() for p, k in enumerate(pl.numel)]
        fs = FlatStep(pl.numel, pl.unit, stage=1, n_ranks=3, init_params=init, guard=256, guard_value=7.0)
        fs.enable_muon(shapes, lr=LR)
        step(fs, grads_for(fs, pl, 3, "bf16", 1))
        assert all((g == 7.0).all() for g in fs.guards())


def test_offsets_beyond_32_bits():
    # matrices of every path behind 2^31 elements of another parameter
    head, mats = 2 ** 31 + 40, [(64, 48), (300, 200), (200, 320), (1, 9)]
    numel = [head] + [r * c for r, c in mats]
    g = torch.Generator(device="cuda").manual_seed(5)
    init = [torch.zeros(head, device="cuda")]
    init += [torch.empty(k, device="cuda").normal_(0.0, 0.02, generator=g) for k in numel[1:]]
    fs = FlatStep(numel, [0] * len(numel), stage=1, n_ranks=1, lr=1e-3, adamw=True, init_params=init)
    del init
    fs.enable_muon([None] + mats, lr=LR, momentum=MU, weight_decay=WD)
    grad = torch.zeros(fs.padded, dtype=torch.bfloat16, device="cuda")
    grad[head:].normal_(0.0, 1e-2, generator=g)
    w0 = fs.master[head:].cpu()
    step(fs, [grad])
    w1, p16 = fs.master[head:].cpu(), fs.param16[head:].cpu()
    assert not fs.master[:head].any() and not fs.exp_avg[:head].any()
    for p, s in enumerate(mats):
        o = fs.param_offset(1 + p)
        at = slice(o - head, o - head + numel[1 + p])
        mine = grad[o:o + numel[1 + p]].float().cpu()
        assert torch.equal(fs.exp_avg[o:o + numel[1 + p]].cpu(), mine)
        want = orthogonalized64(mine.view(s))
        update = (w0[at].double() * (1 - LR * WD) - w1[at].double()) / (LR * muon_scale(*s, "rms"))
        slack = float(w0[at].abs().max()) * 2.0 ** -22 / (LR * muon_scale(*s, "rms")) * np.sqrt(want.numel()) / float(want.norm())
        assert relative(update.view(s), want) <= NS_TOL + slack, s
        assert torch.equal(p16[at], w1[at].bfloat16())
