"""Cases that measure the operators around the orthogonalised (Muon) optimizer step.

Three operators:

* ``ns``    Newton-Schulz orthogonalisation of a stack of matrices (``ops.orthogonalize``);
* ``muon``  one optimizer step over a flat parameter buffer whose matrices take the
  orthogonalised momentum update and whose other parameters stay with AdamW
  (``FlatStep`` after ``enable_muon``);
* ``qk``    norm of the queries and keys of every head with the position rotation in the
  same pass, forward and backward (``ops.qk_norm_rope``, ``ops.qk_norm_rope_backward``).

``run`` takes the plain torch form or, with ``own`` set, the framework's calls; ``exact``
computes the definition in 64 bits.
"""

import math

import torch

own = False

COEFFICIENTS = (3.4445, -4.7750, 2.0315)
STEPS = 5
NS_EPS = 1e-7
LR, WEIGHT_DECAY, MOMENTUM, ADAM_EPS = 2e-4, 0.1, 0.95, 1e-8
# the configuration holds its betas in fp32 and 1 - beta is the difference from that value
BETA1, BETA2 = torch.tensor([0.9, 0.999], dtype=torch.float32).tolist()
QK_EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------------------
# Cases.
# ---------------------------------------------------------------------------
def listed():
    return [
        # one hidden layer of the toy MLP: the smallest call, where latency counts
        {"name": "ns toy 64x64", "op": "ns", "rows": 64, "cols": 64, "batch": 1, "dtype": "fp32"},
        # the key projection of a hidden-2048 layer with 8 of 32 heads for keys, a bf16 gradient
        {"name": "ns k_proj 512x2048", "op": "ns", "rows": 512, "cols": 2048, "batch": 1, "dtype": "bf16"},
        # sizes that no tile divides, several matrices at once
        {"name": "ns odd 777x1301 x3", "op": "ns", "rows": 777, "cols": 1301, "batch": 3, "dtype": "fp32"},
        # the down projections of four hidden-2048 layers: tall matrices, the largest plain orthogonalisation
        {"name": "ns down 8192x2048 x4", "op": "ns", "rows": 8192, "cols": 2048, "batch": 4, "dtype": "fp32"},
        # the whole step of the toy MLP with 4 replicas: launch latency
        {"name": "muon toy mlp n4", "op": "muon", "widths": "32-128-128-64-64-16", "n": 4, "dtype": "bf16"},
        # the whole step of the hidden-1024 Llama-style model, 8 bf16 replicas
        {"name": "muon llama1024 n8", "op": "muon", "hidden": 1024, "inter": 2048, "heads": 16, "kv": 4,
         "layers": 8, "vocab": 1024, "n": 8, "dtype": "bf16"},
        # one decoder layer of the hidden-2048 model, 2 fp32 replicas (gradient accumulation)
        {"name": "muon layer2048 n2 fp32", "op": "muon", "hidden": 2048, "inter": 8192, "heads": 32, "kv": 8,
         "layers": 1, "vocab": 0, "n": 2, "dtype": "fp32"},
        # the whole hidden-2048 model, 8 bf16 replicas: the largest step
        {"name": "muon llama2048 n8", "op": "muon", "hidden": 2048, "inter": 8192, "heads": 32, "kv": 8,
         "layers": 8, "vocab": 40960, "n": 8, "dtype": "bf16"},
        # one new token of one sequence
        {"name": "qk fwd 1 token", "op": "qk", "dir": "fwd", "tokens": 1, "heads": 32, "kv": 8, "dim": 64,
         "rotary": 64, "interleaved": False, "dtype": "bf16"},
        # a training batch of the hidden-2048 model, forward
        {"name": "qk fwd 32768 tokens", "op": "qk", "dir": "fwd", "tokens": 32768, "heads": 32, "kv": 8, "dim": 64,
         "rotary": 64, "interleaved": False, "dtype": "bf16"},
        # ... and its backward with the gradients of both gains
        {"name": "qk bwd 32768 tokens", "op": "qk", "dir": "bwd", "tokens": 32768, "heads": 32, "kv": 8, "dim": 64,
         "rotary": 64, "interleaved": False, "dtype": "bf16"},
        # an odd number of tokens, wide heads with a partial interleaved rotation, fp32
        {"name": "qk bwd 5003 odd fp32", "op": "qk", "dir": "bwd", "tokens": 5003, "heads": 16, "kv": 4, "dim": 80,
         "rotary": 32, "interleaved": True, "dtype": "fp32"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ns", "muon", "qk"])
    if op == "ns":
        while True:
            case = {"op": "ns", "rows": _log_int(rng, 1, 8192), "cols": _log_int(rng, 1, 8192),
                    "batch": _log_int(rng, 1, 16), "dtype": rng.choice(["fp32", "bf16"])}
            if work(case)["flops"] <= work(listed()[3])["flops"]:
                return case
    if op == "muon":
        n, dtype = rng.choice([1, 2, 3, 4, 6, 8, 16]), rng.choice(["bf16", "fp32"])
        if rng.random() < 0.5:  # an MLP of odd widths, one unit per layer
            widths = [_log_int(rng, 9, 1500) for _ in range(rng.randint(3, 6))]
            return {"op": "muon", "widths": "-".join(str(w) for w in widths), "n": n, "dtype": dtype}
        heads = rng.choice([4, 8, 12, 16, 24])
        return {"op": "muon", "hidden": 64 * heads, "inter": 8 * (2 * _log_int(rng, 8 * heads, 16 * heads) + 1),
                "heads": heads, "kv": heads // rng.choice([1, 2, 4]), "layers": rng.randint(1, 6), "vocab": _log_int(rng, 500, 20000),
                "n": n, "dtype": dtype}
    dim = rng.choice([32, 64, 80, 96, 128, 256])
    kv = rng.choice([1, 2, 4, 8])
    return {"op": "qk", "dir": rng.choice(["fwd", "bwd"]), "tokens": _log_int(rng, 1, 16384),
            "heads": kv * rng.choice([1, 3, 4]), "kv": kv, "dim": dim, "rotary": rng.choice([dim, dim // 2]),
            "interleaved": rng.choice([False, True]), "dtype": rng.choice(["bf16", "fp32"])}


def _ns_flops(rows, cols):
    """Five steps over the smaller side m: the symmetric Gram product, its symmetric square, the update of X."""
    m, n = min(rows, cols), max(rows, cols)
    return STEPS * (3.0 * m * m * n + 1.0 * m * m * m)


def work(case):
    if case["op"] == "ns":
        e = case["batch"] * case["rows"] * case["cols"]
        return {"bytes": e * ((4 if case["dtype"] == "fp32" else 2) + 2.0),
                "flops": case["batch"] * _ns_flops(case["rows"], case["cols"])}
    if case["op"] == "muon":
        lay = _layout(case)
        g = case["n"] * (4 if case["dtype"] == "fp32" else 2)
        matrix = sum(r * c for r, c in filter(None, lay["shapes"]))
        # matrices: replicas, momentum and master read, momentum, master and bf16 parameters written;
        # the others also read and write a second moment
        return {"bytes": matrix * (g + 18.0) + (lay["padded"] - matrix) * (g + 26.0),
                "flops": sum(_ns_flops(r, c) for r, c in filter(None, lay["shapes"]))}
    e = case["tokens"] * (case["heads"] + case["kv"]) * case["dim"]
    size = 4 if case["dtype"] == "fp32" else 2
    passes = 2 if case["dir"] == "fwd" else 3
    table = 4.0 * case["tokens"] * case["rotary"]
    return {"bytes": float(passes * e * size + table), "flops": 12.0 * e}


# ---------------------------------------------------------------------------
# Inputs.
# ---------------------------------------------------------------------------
def _layout(case):
    """The flat layout: (rows, cols) of every matrix parameter and None for the others, their offsets, the units
    (each padded to a multiple of the replica count) and the padded total."""
    numel, unit, shapes = [], [], []

    def add(n, u, shape=None):
        numel.append(n)
        unit.append(u)
        shapes.append(shape)

    if "widths" in case:
        w = [int(x) for x in case["widths"].split("-")]
        for i in range(len(w) - 1):
            add(w[i + 1] * w[i], i, (w[i + 1], w[i]))
            add(w[i + 1], i)
    else:
        h, inter, kv, u = case["hidden"], case["inter"], case["hidden"] // case["heads"] * case["kv"], 0
        if case["vocab"]:
            add(case["vocab"] * h, u)  # the embedding stays with AdamW
            u += 1
        for _ in range(case["layers"]):
            for r, c in ((h, h), (kv, h), (kv, h), (h, h), (inter, h), (inter, h), (h, inter)):
                add(r * c, u, (r, c))
            add(h, u)
            add(h, u)
            u += 1
        if case["vocab"]:
            add(h, u)
            add(case["vocab"] * h, u)  # and so does the head
    offsets, base, at = [], 0, 0
    for p, n in enumerate(numel):
        if p and unit[p] != unit[p - 1]:
            base = at = base + -(-(at - base) // case["n"]) * case["n"]
        offsets.append(at)
        at += n
    padded = base + -(-(at - base) // case["n"]) * case["n"]
    return {"numel": numel, "unit": unit, "shapes": shapes, "offsets": offsets, "padded": padded}


def _normal(shape, std, gen):
    return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=gen)


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "ns":
        return {"x": _normal((case["batch"], case["rows"], case["cols"]), 1e-3, gen).to(dtype)}
    if case["op"] == "muon":
        lay = _layout(case)
        real = torch.zeros(lay["padded"], dtype=torch.bool, device="cuda")
        matrix = torch.zeros(lay["padded"], dtype=torch.bool, device="cuda")
        for o, n, s in zip(lay["offsets"], lay["numel"], lay["shapes"]):
            real[o:o + n] = True
            if s is not None:
                matrix[o:o + n] = True
        # momentum of some steps, in the matrices only; pads of the parameters and gradients are zero
        momentum = _normal(lay["padded"], 2e-3, gen).mul_(matrix)
        master = _normal(lay["padded"], 0.02, gen).mul_(real)
        grads = [_normal(lay["padded"], 1e-3, gen).mul_(real).to(dtype) for _ in range(case["n"])]
        return {"master": master, "momentum": momentum, "grads": grads, "others": ~matrix, "lay": lay}
    t, hq, hk, d = case["tokens"], case["heads"], case["kv"], case["dim"]
    # queries and keys as one fused projection leaves them: strided views of its output
    qk = _normal((t, hq + hk, d), 1.0, gen).to(dtype)
    # documents of at most 2048 tokens packed one after another; a sequence's last sixteenth is padding
    index = torch.arange(t, dtype=torch.int32, device="cuda")
    positions = torch.where(index >= t - t // 16, -1, index % 2048).to(torch.int32)
    half = case["rotary"] // 2
    freq = torch.pow(10000.0, -torch.arange(half, dtype=torch.float64, device="cuda") / max(half, 1))
    angle = torch.arange(2048, dtype=torch.float64, device="cuda")[:, None] * freq
    return {"q": qk[:, :hq], "k": qk[:, hq:], "positions": positions,
            "table": torch.cat([angle.cos(), angle.sin()], 1).float(),
            "q_gain": 1.0 + _normal(d, 0.1, gen), "k_gain": 1.0 + _normal(d, 0.1, gen),
            "dq": _normal((t, hq, d), 1.0, gen).to(dtype), "dk": _normal((t, hk, d), 1.0, gen).to(dtype)}


def prepare(case, seed):
    state = dict(_inputs(case, seed), case=case)
    if case["op"] != "muon":
        return state
    lay = state["lay"]
    if own:  # the framework's handle of the same buffers: what a training program keeps from step to step
        from zero_sharded_mixed_flatparameter_gb300.runner import FlatStep
        fs = FlatStep(lay["numel"], lay["unit"], stage=1, n_ranks=case["n"], grad_dtype=case["dtype"], lr=LR,
                      beta1=BETA1, beta2=BETA2, eps=ADAM_EPS, weight_decay=WEIGHT_DECAY, adamw=True,
                      init_params=[state["master"][o:o + n] for o, n in zip(lay["offsets"], lay["numel"])])
        fs.enable_muon(lay["shapes"], lr=LR, momentum=MOMENTUM, weight_decay=WEIGHT_DECAY, nesterov=True, scale="rms",
                       steps=STEPS, coefficients=COEFFICIENTS, eps=NS_EPS)
        fs.exp_avg.copy_(state["momentum"])
        return {"case": case, "fs": fs, "grads": state["grads"]}
    groups = {}
    for o, s in zip(lay["offsets"], lay["shapes"]):
        if s is not None:
            groups.setdefault(s, []).append(o)
    state["groups"] = groups
    state["others"] = state["others"].nonzero().reshape(-1)
    state["second"] = torch.zeros_like(state["master"])
    state["param16"] = state["master"].bfloat16()
    state["t"] = 0
    return state


# ---------------------------------------------------------------------------
# One pass.
# ---------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if op == "ns":
        return _ns_own(state) if own else _orthogonalized(state["x"].float()).bfloat16()
    if op == "muon":
        return _muon_own(state) if own else _muon_plain(state)
    return _qk_own(state) if own else _qk_plain(state)


def _ns_own(state):
    from zero_sharded_mixed_flatparameter_gb300 import ops
    return ops.orthogonalize(state["x"], steps=STEPS, coefficients=COEFFICIENTS, eps=NS_EPS)


def _muon_own(state):
    fs = state["fs"]
    fs.reduce_grads(-1, state["grads"])
    fs.step()
    fs.post_step()
    return {"master": fs.master, "momentum": fs.exp_avg, "second": fs.exp_avg_sq, "param16": fs.param16}


def _qk_own(state):
    from zero_sharded_mixed_flatparameter_gb300 import ops
    case = state["case"]
    args = (state["q"], state["k"], state["q_gain"], state["k_gain"], state["table"], state["positions"])
    if case["dir"] == "fwd":
        q, k = ops.qk_norm_rope(*args, eps=QK_EPS, interleaved=case["interleaved"])
        return {"q": q, "k": k}
    dq, dk, dq_gain, dk_gain = ops.qk_norm_rope_backward(state["dq"], state["dk"], *args, eps=QK_EPS,
                                                         interleaved=case["interleaved"])
    return {"dq": dq, "dk": dk, "dq_gain": dq_gain, "dk_gain": dk_gain}


def _orthogonalized(x):
    """Newton-Schulz steps of a stack of fp32 matrices, over their smaller side."""
    a, b, c = COEFFICIENTS
    tall = x.shape[-2] > x.shape[-1]
    if tall:
        x = x.mT
    x = x / (x.square().sum((-2, -1), keepdim=True).sqrt() + NS_EPS)
    for _ in range(STEPS):
        gram = x @ x.mT
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x.mT if tall else x


def _muon_plain(state):
    state["t"] += 1
    t, others = state["t"], state["others"]
    w, m, v, p16 = state["master"], state["momentum"], state["second"], state["param16"]
    g = sum(x.float() for x in state["grads"]) * (1.0 / state["case"]["n"])
    # AdamW for what is not a matrix (pads are zero and stay zero)
    go = g[others]
    mo = BETA1 * m[others] + (1 - BETA1) * go
    vo = BETA2 * v[others] + (1 - BETA2) * go * go
    m[others], v[others] = mo, vo
    wo = w[others] * (1 - LR * WEIGHT_DECAY)
    w[others] = wo - LR * (mo / (1 - BETA1 ** t)) / ((vo / (1 - BETA2 ** t)).sqrt() + ADAM_EPS)
    # the orthogonalised momentum for the matrices, those of one shape together
    for (r, c), offsets in state["groups"].items():
        parts = [slice(o, o + r * c) for o in offsets]
        gm = torch.stack([g[s] for s in parts]).view(-1, r, c)
        mom = MOMENTUM * torch.stack([m[s] for s in parts]).view(-1, r, c) + gm
        update = _orthogonalized(gm + MOMENTUM * mom) * (LR * 0.2 * math.sqrt(max(r, c)))
        wm = torch.stack([w[s] for s in parts]).view(-1, r, c) * (1 - LR * WEIGHT_DECAY) - update
        for s, mi, wi in zip(parts, mom, wm):
            m[s], w[s] = mi.view(-1), wi.view(-1)
    p16.copy_(w)
    return {"master": w, "momentum": m, "second": v, "param16": p16}


def _rotation(state, dtype):
    """cos and sin of every token's position (shape tokens x 1 x rotary/2) and which tokens are padding."""
    position = state["positions"].long()
    row = state["table"].to(dtype)[position.clamp(min=0)][:, None]
    half = state["case"]["rotary"] // 2
    return row[..., :half], row[..., half:], (position < 0)[:, None, None]


def _pairs(state, x):
    """The two halves of every rotated pair, and the part that is not rotated."""
    rotary = state["case"]["rotary"]
    if state["case"]["interleaved"]:
        return x[..., 0:rotary:2], x[..., 1:rotary:2], x[..., rotary:]
    return x[..., :rotary // 2], x[..., rotary // 2:rotary], x[..., rotary:]


def _unpaired(state, first, second, rest):
    if state["case"]["interleaved"]:
        return torch.cat([torch.stack([first, second], -1).flatten(-2), rest], -1)
    return torch.cat([first, second, rest], -1)


def _qk_plain(state):
    cos, sin, padding = _rotation(state, torch.float32)

    def forward(x, gain):
        x32 = x.float()
        y = x32 * torch.rsqrt(x32.square().mean(-1, keepdim=True) + QK_EPS) * gain
        first, second, rest = _pairs(state, y)
        y = _unpaired(state, first * cos - second * sin, second * cos + first * sin, rest)
        return y.masked_fill(padding, 0.0).to(x.dtype)

    def backward(dy, x, gain):
        x32 = x.float()
        rstd = torch.rsqrt(x32.square().mean(-1, keepdim=True) + QK_EPS)
        first, second, rest = _pairs(state, dy.float().masked_fill(padding, 0.0))
        h = _unpaired(state, first * cos + second * sin, second * cos - first * sin, rest)
        normed = (x32 * rstd).masked_fill(padding, 0.0)
        dgain = (h * normed).sum((0, 1))
        h = h * gain
        return (rstd * (h - normed * (h * normed).mean(-1, keepdim=True))).masked_fill(padding, 0.0).to(x.dtype), dgain

    if state["case"]["dir"] == "fwd":
        return {"q": forward(state["q"], state["q_gain"]), "k": forward(state["k"], state["k_gain"])}
    dq, dq_gain = backward(state["dq"], state["q"], state["q_gain"])
    dk, dk_gain = backward(state["dk"], state["k"], state["k_gain"])
    return {"dq": dq, "dk": dk, "dq_gain": dq_gain, "dk_gain": dk_gain}


# ---------------------------------------------------------------------------
# The definitions in 64 bits.
# ---------------------------------------------------------------------------
def _ns64(x):
    """One matrix: five steps X <- X (a I + b X'X + c (X'X)^2), the products over the smaller side."""
    if x.shape[0] < x.shape[1]:
        return _ns64(x.T).T
    a, b, c = COEFFICIENTS
    x = x / (torch.linalg.matrix_norm(x) + NS_EPS)
    for _ in range(STEPS):
        s = x.T @ x
        p = torch.addmm(s, s, s, beta=b, alpha=c)
        p.diagonal().add_(a)
        x = x @ p
    return x


def exact(case, seed):
    if work(case)["flops"] > 6e12 and case["op"] == "muon":
        return None  # over 20 seconds of 64-bit products
    data = _inputs(case, seed)
    if case["op"] == "ns":
        return torch.stack([_ns64(x.double()) for x in data["x"]])
    if case["op"] == "muon":
        lay = data["lay"]
        w, m = data["master"].double(), data["momentum"].double()
        v = torch.zeros_like(w)
        g = torch.zeros_like(w)
        for x in data["grads"]:
            g += x.double() / case["n"]
        w *= 1 - LR * WEIGHT_DECAY
        step = LR * g / (g.abs() + ADAM_EPS)  # the first AdamW step from zero moments, bias corrected
        w -= torch.where(data["others"], step, 0.0)
        v += torch.where(data["others"], (1 - BETA2) * g * g, 0.0)
        m = torch.where(data["others"], (1 - BETA1) * g, MOMENTUM * m + g)
        for o, s in zip(lay["offsets"], lay["shapes"]):
            if s is not None:
                at = slice(o, o + s[0] * s[1])
                update = _ns64((g[at] + MOMENTUM * m[at]).view(s))
                w[at] -= (LR * 0.2 * math.sqrt(max(s)) * update).reshape(-1)
        return {"master": w, "momentum": m, "second": v, "param16": w}
    # queries and keys: the rotation as a product of complex numbers, the gradients by reverse differentiation
    live = data["positions"] >= 0
    rotary, half = case["rotary"], case["rotary"] // 2
    row = data["table"].double()[data["positions"].long() * live]
    turn = torch.complex(row[:, :half], row[:, half:])[:, None]

    def definition(x, gain):
        y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + QK_EPS) * gain
        if case["interleaved"]:
            z = torch.complex(y[..., 0:rotary:2], y[..., 1:rotary:2]) * turn
            z = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(y[..., :half], y[..., half:rotary]) * turn
            z = torch.cat([z.real, z.imag], -1)
        return torch.cat([z, y[..., rotary:]], -1) * live[:, None, None]

    out = {}
    for name in ("q", "k"):
        x, gain = data[name].double().requires_grad_(), data[name + "_gain"].double().requires_grad_()
        y = definition(x, gain)
        if case["dir"] == "fwd":
            out[name] = y.detach()
        else:
            out["d" + name], out["d" + name + "_gain"] = torch.autograd.grad(y, (x, gain), data["d" + name].double())
    return out
