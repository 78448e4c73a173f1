"""Cases that measure the operators between a training step's matrix products.

Three operators:

* ``norm``   layer norm over the hidden dimension (also without centring), forward and backward
  with the gradients of weight and bias, and both with the input kept in 8 bits in between
  (``ops.layer_norm``, ``ops.layer_norm_backward``);
* ``pack``   activations to 8 bits with a power-of-two scale for every 32 columns, and back
  (``ops.pack_activations``, ``ops.unpack_activations``);
* ``embed``  embedding lookup with a factor, and the table's gradient by sorted tokens
  (``ops.embedding``, ``ops.embedding_backward``).

``run`` takes the plain torch form or, with ``own`` set, the framework's calls; ``exact``
computes the definition in 64 bits.
"""

import math

import torch

own = False

EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
FORMATS = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
GROUP = 32


# ---------------------------------------------------------------------------
# Cases.
# ---------------------------------------------------------------------------
def listed():
    return [
        # the norm before the projections for one new token: the smallest call, where latency counts
        {"name": "norm fwd 1 row", "op": "norm", "dir": "fwd", "rows": 1, "cols": 2048, "center": False, "bias": False,
         "dtype": "bf16", "pack": ""},
        # a training batch of the hidden-2048 model, weight and bias
        {"name": "norm fwd 32768x2048", "op": "norm", "dir": "fwd", "rows": 32768, "cols": 2048, "center": True,
         "bias": True, "dtype": "bf16", "pack": ""},
        # ... and its backward with the gradients of both
        {"name": "norm bwd 32768x2048", "op": "norm", "dir": "bwd", "rows": 32768, "cols": 2048, "center": True,
         "bias": True, "dtype": "bf16", "pack": ""},
        # sizes that no vector divides, fp32 gradients
        {"name": "norm bwd odd 5003x1301 fp32", "op": "norm", "dir": "bwd", "rows": 5003, "cols": 1301, "center": True,
         "bias": True, "dtype": "fp32", "pack": ""},
        # a layer's first norm in a training step that keeps its input in 8 bits: forward, later backward from those
        {"name": "norm kept 16384x2048", "op": "norm", "dir": "both", "rows": 16384, "cols": 2048, "center": False,
         "bias": False, "dtype": "bf16", "pack": "e4m3"},
        # a micro-batch's block input of the hidden-1024 model kept in 8 bits, and restored
        {"name": "pack 2048x1024", "op": "pack", "rows": 2048, "cols": 1024, "dtype": "bf16", "pack": "e4m3"},
        # an odd width in fp32, to whole numbers
        {"name": "pack odd 4099x777 fp32", "op": "pack", "rows": 4099, "cols": 777, "dtype": "fp32", "pack": "int8"},
        # the input of the hidden-2048 model's down projection over a training batch: the largest
        {"name": "pack 32768x8192", "op": "pack", "rows": 32768, "cols": 8192, "dtype": "bf16", "pack": "e4m3"},
        # one new token
        {"name": "embed fwd 1 token", "op": "embed", "dir": "fwd", "tokens": 1, "vocab": 40960, "dim": 2048,
         "scale": 1.0, "dtype": "bf16", "ids": "int64"},
        # a training batch, lookup with a factor
        {"name": "embed fwd 32768 tokens", "op": "embed", "dir": "fwd", "tokens": 32768, "vocab": 40960, "dim": 2048,
         "scale": 45.25, "dtype": "bf16", "ids": "int64"},
        # ... and the gradient of the whole table
        {"name": "embed bwd 32768 tokens", "op": "embed", "dir": "bwd", "tokens": 32768, "vocab": 40960, "dim": 2048,
         "scale": 45.25, "dtype": "bf16", "ids": "int64"},
        # a small vocabulary, every row in use many times over, odd sizes
        {"name": "embed bwd odd 5003 fp32", "op": "embed", "dir": "bwd", "tokens": 5003, "vocab": 1009, "dim": 321,
         "scale": 1.0, "dtype": "fp32", "ids": "int32"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _odd(rng, n):
    """Half of the sizes are whole vectors, the others what comes."""
    return max(8, n // 8 * 8) if rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["norm", "norm", "pack", "embed", "embed"])
    dtype = rng.choice(["bf16", "fp32"])
    while True:
        if op == "norm":
            direction = rng.choice(["fwd", "bwd", "both"])
            case = {"op": "norm", "dir": direction, "rows": _log_int(rng, 1, 32768), "cols": _odd(rng, _log_int(rng, 1, 8192)),
                    "center": rng.choice([True, False]), "bias": rng.choice([True, False]), "dtype": dtype,
                    "pack": rng.choice(["e4m3", "int8"]) if direction == "both" else ""}
        elif op == "pack":
            case = {"op": "pack", "rows": _log_int(rng, 1, 32768), "cols": _odd(rng, _log_int(rng, 1, 8192)),
                    "dtype": dtype, "pack": rng.choice(["e4m3", "int8"])}
        else:
            case = {"op": "embed", "dir": rng.choice(["fwd", "bwd"]), "tokens": _log_int(rng, 1, 32768),
                    "vocab": _log_int(rng, 2, 65536), "dim": _odd(rng, _log_int(rng, 1, 2048)),
                    "scale": rng.choice([1.0, 45.25]), "dtype": dtype, "ids": rng.choice(["int32", "int64"])}
        if work(case)["bytes"] <= work(listed()[2])["bytes"]:
            return case


def _used_rows(case):
    """How many rows of the table the tokens of `_ids` use, on average."""
    v, live = case["vocab"], case["tokens"] - case["tokens"] // 16
    edge = torch.arange(1, v + 2, dtype=torch.float64).log() / math.log(v + 1)
    return float((1 - (1 - edge.diff()).pow(live)).sum())


def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "embed":
        live = case["tokens"] - case["tokens"] // 16
        ids = case["tokens"] * (8 if case["ids"] == "int64" else 4)
        if case["dir"] == "fwd":
            return {"bytes": (_used_rows(case) + case["tokens"]) * case["dim"] * size + ids,
                    "flops": float(case["tokens"] * case["dim"])}
        return {"bytes": (live + case["vocab"]) * float(case["dim"] * size) + ids, "flops": 2.0 * live * case["dim"]}
    e = case["rows"] * case["cols"]
    kept = e + case["rows"] * -(-case["cols"] // GROUP)  # codes and scales
    if case["op"] == "pack":
        return {"bytes": 2.0 * (e * size + kept), "flops": 4.0 * e}
    # weight and bias are fp32, and so are their gradients; the forward pass hands two statistics of a row to the backward
    vectors = 4.0 * case["cols"] * (2 if case["bias"] else 1)
    fwd, bwd = 2 * e * size + 8.0 * case["rows"] + vectors, 3 * e * size + 8.0 * case["rows"] + vectors + 4.0 * case["cols"]
    if case["dir"] == "both":  # the backward pass reads the kept form instead of the input
        return {"bytes": fwd + bwd - e * size + 2.0 * kept, "flops": 28.0 * e}
    return {"bytes": fwd, "flops": 9.0 * e} if case["dir"] == "fwd" else {"bytes": bwd, "flops": 15.0 * e}


# ---------------------------------------------------------------------------
# Inputs.
# ---------------------------------------------------------------------------
def _normal(shape, std, gen):
    return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=gen)


def _activations(rows, cols, gen, dtype):
    """Hidden states: rows of different size, a few columns that are far larger than the others, a mean."""
    x = _normal((rows, cols), 1.0, gen)
    x *= 0.5 + _normal((rows, 1), 1.0, gen).abs()
    x[:, 5::419] *= 25.0
    return x.add_(0.2).to(dtype)


def _ids(case, gen):
    """Ids of a text: the probability falls with the id as 1 / id; the last sixteenth is padding."""
    t, v = case["tokens"], case["vocab"]
    u = torch.empty(t, dtype=torch.float64, device="cuda").uniform_(0.0, 1.0, generator=gen)
    ids = (torch.exp(u * math.log(v + 1)).floor().long() - 1).clamp_(0, v - 1)
    ids[t - t // 16:] = -1
    return ids.to(torch.int32 if case["ids"] == "int32" else torch.int64)


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "pack":
        return {"x": _activations(case["rows"], case["cols"], gen, dtype)}
    if case["op"] == "embed":
        data = {"ids": _ids(case, gen)}
        if case["dir"] == "fwd":
            data["table"] = _normal((case["vocab"], case["dim"]), 0.02, gen).to(dtype)
        else:
            data["dy"] = _normal((case["tokens"], case["dim"]), 1e-3, gen).to(dtype)
        return data
    rows, cols = case["rows"], case["cols"]
    data = {"x": _activations(rows, cols, gen, dtype), "weight": 1.0 + _normal(cols, 0.1, gen),
            "bias": _normal(cols, 0.1, gen) if case["bias"] else None}
    if case["dir"] != "fwd":
        data["dy"] = _normal((rows, cols), 1e-3, gen).to(dtype)
    if case["dir"] == "bwd":  # what the forward pass has handed on
        data["stats"] = torch.stack(_moments(data["x"].double(), case["center"]), 1).float()
    return data


def _moments(x, center):
    mean = x.mean(1) if center else torch.zeros_like(x[:, 0])
    return mean, torch.rsqrt((x - mean[:, None]).square().mean(1) + EPS)


def prepare(case, seed):
    return dict(_inputs(case, seed), case=case)


# ---------------------------------------------------------------------------
# One pass.
# ---------------------------------------------------------------------------
def run(state):
    case = state["case"]
    if case["op"] == "norm":
        return _norm_own(state, case) if own else _norm_plain(state, case)
    if case["op"] == "pack":
        return _pack_own(state, case) if own else _packed_values(state["x"], case["pack"]).to(state["x"].dtype)
    return _embed_own(state, case) if own else _embed_plain(state, case)


def _norm_own(state, case):
    from zero_sharded_mixed_flatparameter_gb300 import ops
    x, weight, bias, center = state["x"], state["weight"], state["bias"], case["center"]
    if case["dir"] == "fwd":
        y, stats = ops.layer_norm(x, weight, bias, eps=EPS, center=center)
        return {"y": y, "stats": stats}
    out = {}
    stats = state.get("stats")
    if case["dir"] == "both":
        out["y"], stats, x = ops.layer_norm(x, weight, bias, eps=EPS, center=center, pack=FORMATS[case["pack"]])
    out["dx"], out["dweight"], dbias = ops.layer_norm_backward(state["dy"], x, weight, stats, center=center,
                                                               bias=case["bias"])
    if case["bias"]:
        out["dbias"] = dbias
    return out


def _pack_own(state, case):
    from zero_sharded_mixed_flatparameter_gb300 import ops
    return ops.unpack_activations(ops.pack_activations(state["x"], FORMATS[case["pack"]]))


def _embed_own(state, case):
    from zero_sharded_mixed_flatparameter_gb300 import ops
    if case["dir"] == "fwd":
        return ops.embedding(state["ids"], state["table"], scale=case["scale"])
    return ops.embedding_backward(state["dy"], state["ids"], case["vocab"], scale=case["scale"])


def _power(exponent):
    """2 to whole exponents of fp32's normal range, exactly."""
    return (exponent + 127 << 23).view(torch.float32)


def _packed_values(x, form):
    """The values that the 8-bit form of x stands for, fp32: a group's scale is the smallest power of two that keeps
    its largest entry within the format; a group that is not finite reads as NaN."""
    rows, cols = x.shape
    groups = torch.nn.functional.pad(x.float(), (0, -cols % GROUP)).view(rows, -1, GROUP)
    largest = groups.abs().amax(-1, keepdim=True)
    mantissa, exponent = torch.frexp(largest)
    if form == "e4m3":
        exponent = exponent - 9 + (mantissa > 0.875).int()
    else:
        exponent = exponent - 7 + (mantissa > 127 / 128).int()
    exponent = exponent.clamp(min=-126)
    scaled = groups * _power(-exponent)
    codes = scaled.to(torch.float8_e4m3fn).float() if form == "e4m3" else scaled.round()
    values = (codes * _power(exponent)).masked_fill(~largest.isfinite(), math.nan)
    return values.view(rows, -1)[:, :cols]


def _norm_plain(state, case):
    x, dtype, center = state["x"].float(), state["x"].dtype, case["center"]
    weight, bias, out = state["weight"], state["bias"], {}
    if "stats" in state:
        mean, rstd = state["stats"][:, :1], state["stats"][:, 1:]
    else:
        mean, rstd = (s[:, None] for s in _moments(x, center))
        y = (x - mean) * rstd * weight
        out["y"] = (y if bias is None else y + bias).to(dtype)
        if case["dir"] == "fwd":
            out["stats"] = torch.cat([mean, rstd], 1)
            return out
    if case["dir"] == "both":
        x = _packed_values(state["x"], case["pack"])
    dy = state["dy"].float()
    normed = (x - mean) * rstd
    g = dy * weight
    dx = g - normed * (g * normed).mean(1, keepdim=True)
    if center:
        dx = dx - g.mean(1, keepdim=True)
    out["dx"] = (dx * rstd).to(dtype)
    out["dweight"] = (dy * normed).sum(0)
    if bias is not None:
        out["dbias"] = dy.sum(0)
    return out


def _embed_plain(state, case):
    ids, scale = state["ids"].long(), case["scale"]
    live = ids >= 0
    if case["dir"] == "fwd":
        table = state["table"]
        rows = table[ids.clamp(min=0)].float() * scale
        return rows.masked_fill(~live[:, None], 0.0).to(table.dtype)
    dy = state["dy"]
    grad = torch.zeros(case["vocab"] + 1, case["dim"], device="cuda")  # the last row takes the padding
    grad.index_add_(0, torch.where(live, ids, case["vocab"]), dy.float())
    return (grad[:-1] * scale).to(dy.dtype)


# ---------------------------------------------------------------------------
# The definitions in 64 bits.
# ---------------------------------------------------------------------------
def _power64(exponent):
    return (exponent.long() + 1023 << 52).view(torch.float64)


def _quantised64(x, form):
    """Groups one after another: the scale by its logarithm, the codes by their distance to the next value."""
    limit = 448.0 if form == "e4m3" else 127.0
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for at in range(0, x.shape[1], GROUP):
        g = x[:, at:at + GROUP].double()
        top = g.abs().max(dim=1, keepdim=True).values
        k = torch.where(top > 0, torch.ceil(torch.log2(top / limit)), -126.0)
        # the logarithm's rounding: the smallest power that keeps the largest entry within the limit
        k = torch.where(top > limit * _power64(k), k + 1, k)
        k = torch.where(top <= limit * _power64(k - 1), k - 1, k).clamp(min=-126)
        v = g / _power64(k)
        if form == "e4m3":
            step = _power64(v.abs().clamp(min=2.0 ** -6).log2().floor() - 3)
            out[:, at:at + GROUP] = (v / step).round() * step * _power64(k)
        else:
            out[:, at:at + GROUP] = v.round() * _power64(k)
    return out


def exact(case, seed):
    data = _inputs(case, seed)
    if case["op"] == "pack":
        return _quantised64(data["x"], case["pack"])
    if case["op"] == "embed":
        ids = data["ids"].long()
        live = (ids >= 0).nonzero().reshape(-1)
        if case["dir"] == "fwd":
            out = torch.zeros(case["tokens"], case["dim"], dtype=torch.float64, device="cuda")
            out[live] = case["scale"] * data["table"].double()[ids[live]]
            return out
        # by prefix sums over the tokens in the order of their ids, some columns at a time
        order = live[torch.argsort(ids[live], stable=True)]
        ends = torch.bincount(ids[live], minlength=case["vocab"]).cumsum(0)
        out = torch.empty(case["vocab"], case["dim"], dtype=torch.float64, device="cuda")
        for at in range(0, case["dim"], 256):
            sums = torch.nn.functional.pad(data["dy"][order, at:at + 256].double().cumsum(0), (0, 0, 1, 0))
            out[:, at:at + 256] = case["scale"] * (sums[ends] - sums[torch.nn.functional.pad(ends[:-1], (1, 0))])
        return out
    # the norm: gradients by reverse differentiation
    center = case["center"]
    x = data["x"].double()
    weight = data["weight"].double().requires_grad_()
    bias = data["bias"].double().requires_grad_() if case["bias"] else None
    out = {}
    if case["dir"] != "both":
        x.requires_grad_()
    d = x - x.mean(1, keepdim=True) if center else x
    rstd = 1 / torch.sqrt((d * d).sum(1, keepdim=True) / x.shape[1] + EPS)
    y = d * rstd * weight
    if bias is not None:
        y = y + bias
    if case["dir"] == "fwd":
        mean = (x - d)[:, :1] if center else torch.zeros_like(rstd)
        return {"y": y.detach(), "stats": torch.cat([mean, rstd], 1).detach()}
    dy = data["dy"].double()
    if case["dir"] == "bwd":
        grads = torch.autograd.grad(y, [x, weight] + ([bias] if case["bias"] else []), dy)
        return dict(zip(("dx", "dweight", "dbias"), grads))
    # from the kept form: its entries in place of the input's, the statistics still the input's
    out["y"] = y.detach()
    mean = x.mean(1, keepdim=True) if center else 0.0
    rstd = rstd.detach()
    normed = (_quantised64(data["x"], case["pack"]) - mean) * rstd
    g = dy * weight.detach()
    out["dx"] = rstd * (g - (g.mean(1, keepdim=True) if center else 0.0) - normed * (g * normed).mean(1, keepdim=True))
    out["dweight"] = torch.einsum("rc,rc->c", dy, normed)
    if case["bias"]:
        out["dbias"] = dy.sum(0)
    return out
