"""The Muon step's contracts on matrices with both sides above 128 (momentum,
normalisation and products as launches of their own), and the forms and batches
that their sizes lead to."""

import numpy as np
import pytest
import torch

import oracle
import synth_inputs as si
from gpu_common import ensure_built
from muon_reference import NS_TOL, muon_scale, orthogonalized64, relative
from test_gpu_muon import LR, MU, WD, check_matrices, grads_for, make, mlp, reduced, snapshot, step
from zero_sharded_mixed_flatparameter_gb300.runner import FlatStep

pytestmark = pytest.mark.gpu

NAMES = ("master", "exp_avg", "exp_avg_sq", "param16")
# matrices of any alignment (odd sizes, odd replica counts pad to anything) and of whole vectors
ODD, EVEN = [150, 301, 200, 9], [160, 304, 208, 16]


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def params(shapes):
    """A unit per matrix, each with a vector of its rows behind it."""
    pl = si.ParamList("matrices")
    out = []
    for i, s in enumerate(shapes):
        pl.add(f"m{i}", s[0] * s[1], i)
        pl.add(f"b{i}", s[0], i)
        out += [s, None]
    return pl, out


def equal(a, b):
    for name in NAMES:
        assert torch.equal(getattr(a, name), getattr(b, name)), name


@pytest.mark.parametrize("widths,n", [(ODD, 3), (EVEN, 4)])
@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("scale", ["rms", "aspect"])
def test_variants(nesterov, scale, widths, n):
    pl, shapes = mlp(widths)
    fs = make(pl, shapes, n, nesterov=nesterov, scale=scale, weight_decay=0.0)
    for t in range(2):
        grads = grads_for(fs, pl, n, "bf16", t + 5)
        before = snapshot(fs)
        step(fs, grads)
        check_matrices(fs, pl, shapes, before, reduced(grads), nesterov, scale, wd=0.0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("widths,n", [(ODD, 5), (EVEN, 8)])
def test_stages_agree(widths, n, dtype):
    # padding moves every matrix to another alignment; the results stay bit for bit
    pl, shapes = mlp(widths)
    state = []
    for stage in (0, 1, 2, 3):
        fs = make(pl, shapes, n, stage=stage, dtype=dtype)
        for t in range(2):
            step(fs, grads_for(fs, pl, n, dtype, t + 1))
        state.append([torch.cat([x[fs.param_offset(p):fs.param_offset(p) + k] for p, k in enumerate(pl.numel)])
                      for x in (fs.master, fs.exp_avg, fs.exp_avg_sq, fs.param16)])
    for other in state[1:]:
        for a, b in zip(state[0], other):
            assert torch.equal(a, b)


@pytest.mark.parametrize("widths", [ODD, EVEN])
def test_unit_buffers_of_any_alignment(widths):
    pl, shapes = mlp(widths)
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
    equal(fs, whole)


@pytest.mark.parametrize("widths,n", [(ODD, 3), (EVEN, 4)])
@pytest.mark.parametrize("keep", [False, True])
def test_clipped(keep, widths, n):
    pl, shapes = mlp(widths)
    fs = make(pl, shapes, n)
    grads = grads_for(fs, pl, n, "bf16", 2)
    before = snapshot(fs)
    fs.reduce_grads(-1, grads)
    fs.clip_grad_norm(0.05, keep_reduced=keep)
    fs.step()
    norm = fs.grad_norm()
    fs.post_step()
    assert norm > 0.05
    check_matrices(fs, pl, shapes, before, reduced(grads, torch.tensor(oracle.clip_coef(norm, 0.05))))


@pytest.mark.parametrize("widths", [ODD, EVEN])
def test_clip_kept_is_bit_identical(widths):
    pl, shapes = mlp(widths)
    a, b = make(pl, shapes, 4), make(pl, shapes, 4)
    for t in range(2):
        grads = grads_for(a, pl, 4, "bf16", t + 1)
        step(a, grads, clip=0.05)
        step(b, grads, clip=0.05, keep=True)
    equal(a, b)


@pytest.mark.parametrize("shapes", [[(150, 300), (301, 150), (20, 60)],  # thin ones beside them
                                    [(200, 320)],                        # one stack by itself
                                    [(30, 2000), (300, 200)]],           # both want the workspace
                         ids=str)
def test_captured_steps_and_their_end(shapes):
    pl, shapes = params(shapes)
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
        equal(fs, eager)
    fs.disable_capturable()


@pytest.mark.parametrize("widths,n", [(ODD, 3), (EVEN, 2)])
def test_nonfinite_count_and_zero_gradients(widths, n):
    pl, shapes = mlp(widths)
    fs = make(pl, shapes, n)
    counter = torch.zeros(1, dtype=torch.int64, device="cuda")
    fs.count_nonfinite(counter)
    zero = [torch.zeros(fs.padded, dtype=torch.bfloat16, device="cuda") for _ in range(n)]
    before = snapshot(fs)
    step(fs, zero)
    assert counter.item() == 0
    at = slice(0, pl.numel[0])
    decay = torch.tensor(1 - np.float64(np.float32(LR)) * np.float64(np.float32(WD)), dtype=torch.float64).float()
    assert torch.equal(fs.master.cpu()[at], before[0][at] * decay), "no gradient, no momentum: decay alone"
    zero[0][3] = float("nan")
    zero[1][pl.numel[0] - 1] = float("inf")
    zero[0][pl.numel[0] + 2] = float("inf")  # not of a matrix: AdamW's part counts, too
    step(fs, zero)
    assert counter.item() == 3
    assert fs.master[at].isnan().all() and fs.master[fs.param_offset(2):fs.param_offset(2) + pl.numel[2]].isfinite().all()


def test_checkpoint_resumes():
    pl, shapes = mlp(ODD)
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


MANY = {
    "14 shapes in two batches": [(130 + 10 * i, 320 - 12 * i) for i in range(14)],
    "70 equal ones": [(130, 140)] * 70,
    "workspace before and after": [(30, 2000), (300, 200), (2000, 30), (200, 300)],
    "split by two": [(1024, 1024), (9, 30)],
    "split by eight beside others": [(512, 2048), (5, 5)],
    "pairs": [(2048, 2048), (2048, 2048), (700, 900)],
}


@pytest.mark.parametrize("name", MANY)
def test_batches_and_forms(name):
    pl, shapes = params(MANY[name])
    fs, again = make(pl, shapes, 2), make(pl, shapes, 2)
    timeouts = fs.kernel_timeouts()
    for t in range(2):
        grads = grads_for(fs, pl, 2, "bf16", t + 3)
        before = snapshot(fs)
        step(fs, grads)
        if t == 0 or len(shapes) < 20:
            check_matrices(fs, pl, shapes, before, reduced(grads))
        step(again, grads)
        equal(fs, again)
    assert fs.kernel_timeouts() == timeouts


def test_steps_one_after_another_without_waiting():
    # nothing waits between the steps; the results are those of steps with a wait after each
    pl, shapes = params([(30, 2000), (300, 200), (160, 304), (20, 33), (520, 260)])
    a, b = make(pl, shapes, 3), make(pl, shapes, 3)
    grads = [grads_for(a, pl, 3, "bf16", t + 1) for t in range(6)]
    torch.cuda.synchronize()
    for g in grads:
        step(a, g, clip=0.05)
    for g in grads:
        step(b, g, clip=0.05)
        torch.cuda.synchronize()
    equal(a, b)


def test_batches_that_use_the_workspace_again():
    # 2^27 elements at once at most: two of the large matrices, then the third, then the others
    large, small = (192, 1 << 18), [(300, 200), (260, 131)]
    mats = [large, large, small[0], large, small[1]]
    numel = [r * c for r, c in mats]
    gen = torch.Generator(device="cuda").manual_seed(9)
    init = [torch.empty(k, device="cuda").normal_(0.0, 0.02, generator=gen) for k in numel]
    fs = FlatStep(numel, [0] * len(mats), stage=1, n_ranks=1, lr=1e-3, adamw=True, init_params=init)
    fs.enable_muon(mats, lr=LR, momentum=MU, weight_decay=WD)
    timeouts = fs.kernel_timeouts()
    grad = torch.empty(fs.padded, dtype=torch.bfloat16, device="cuda").normal_(0.0, 1e-2, generator=gen)
    step(fs, [grad])
    for p, s in enumerate(mats):
        at = slice(fs.param_offset(p), fs.param_offset(p) + numel[p])
        g = grad[at].float()
        assert torch.equal(fs.exp_avg[at], g), p
        want = orthogonalized64((g + torch.tensor(MU, device="cuda") * g).view(s))
        size = LR * muon_scale(*s, "rms")
        update = (init[p].double() * (1 - LR * WD) - fs.master[at].double()) / size
        slack = float(init[p].abs().max()) * 2.0 ** -22 / size * np.sqrt(want.numel()) / float(want.norm())
        assert relative(update.view(s), want) <= NS_TOL + slack, p
        assert torch.equal(fs.param16[at], fs.master[at].bfloat16())
    assert fs.kernel_timeouts() == timeouts
