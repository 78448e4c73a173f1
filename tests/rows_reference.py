"""Plain 64-bit forms that the tests of the layer norm, of the 8-bit form of
activations and of the embedding compare with, written from the formulas with
torch on the CPU."""

from __future__ import annotations

import math

import torch

GROUP = 32
E4M3, INT8 = torch.float8_e4m3fn, torch.int8
U32 = 2.0 ** -24  # half a step of fp32, relative


def half_step(dtype: torch.dtype) -> float:
    return torch.finfo(dtype).eps / 2


def assert_near(got: torch.Tensor, want: torch.Tensor, slack) -> None:
    """|got - want| within half a step of got's type plus `slack`, element by
    element; NaN and infinities where want has them."""
    assert got.shape == want.shape, (got.shape, want.shape)
    wrong_type = half_step(got.dtype)
    tiny = torch.finfo(got.dtype).smallest_normal * wrong_type  # a subnormal's half step
    got, want = got.detach().double().cpu(), want.detach().double()
    finite = want.isfinite()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got[~finite].nan_to_num(), want[~finite].nan_to_num())
    off = (got - want).abs()
    room = wrong_type * want.abs() + torch.as_tensor(slack, dtype=torch.float64).broadcast_to(want.shape) + tiny
    bad = finite & (off > room)
    assert not bad.any(), (int(bad.sum()), float((off / room)[finite].max()), bad.nonzero()[:3].tolist())


def moments64(x: torch.Tensor, eps: float, center: bool):
    x = x.double()
    mean = x.mean(-1, keepdim=True) if center else torch.zeros_like(x[..., :1])
    return mean, 1 / torch.sqrt((x - mean).square().mean(-1, keepdim=True) + eps)


def norm64(x, weight, bias, eps, center):
    """y and the room for fp32 arithmetic in it.

    mean: a sum over at most 8 + 5 + 32 additions in a row, off by 45 half
    steps of mean|x|; the squares' sum likewise, half of it in 1 / sqrt, which is
    itself off by 2^-22, and three more products: below 64 half steps of the
    terms that make up y.
    """
    mean, rstd = moments64(x, eps, center)
    x = x.double()
    w = torch.ones(x.shape[-1], dtype=torch.float64) if weight is None else weight.double()
    b = torch.zeros(x.shape[-1], dtype=torch.float64) if bias is None else bias.double()
    y = (x - mean) * rstd * w + b
    room = 64 * U32 * ((w * rstd).abs() * ((x - mean).abs() + (x.abs().mean(-1, keepdim=True) if center else 0)) + b.abs())
    return y, room


def norm_backward64(dy, x, weight, stats, center):
    """(dx, dweight, dbias), each with the room for fp32 arithmetic in it, from
    given statistics.

    dx: xn is off by 2 half steps of itself, g by one, the two means by 47 of the
    mean of their magnitudes.  Column sums: a CTA's rows in a row (a share of
    1/152), then 32 warps' shares of the CTAs, then 32 more: below 128 additions
    for up to 4000 rows.
    """
    dy, x = dy.double().reshape(-1, dy.shape[-1]), x.double().reshape(-1, x.shape[-1])
    mean, rstd = stats.double()[:, :1], stats.double()[:, 1:]
    w = torch.ones(x.shape[-1], dtype=torch.float64) if weight is None else weight.double()
    xn = (x - mean) * rstd
    g = dy * w
    m2 = (g * xn).mean(1, keepdim=True)
    dx = g - xn * m2
    room = g.abs() + xn.abs() * (g * xn).abs().mean(1, keepdim=True)
    if center:
        dx = dx - g.mean(1, keepdim=True)
        room = room + g.abs().mean(1, keepdim=True)
    return ((rstd * dx, 64 * U32 * rstd.abs() * room), ((dy * xn).sum(0), 128 * U32 * (dy * xn).abs().sum(0)),
            (dy.sum(0), 128 * U32 * dy.abs().sum(0)))


def pack64(x: torch.Tensor, form: torch.dtype):
    """(codes' values, exponents, values) of a matrix, group by group."""
    limit = 448.0 if form == E4M3 else 127.0
    rows, cols = x.shape
    groups = -(-cols // GROUP)
    padded = torch.zeros(rows, groups * GROUP, dtype=torch.float64)
    padded[:, :cols] = x.double()
    codes = torch.zeros_like(padded)
    exponents = torch.zeros(rows, groups, dtype=torch.int64)
    values = torch.zeros_like(padded)
    for r in range(rows):
        for j in range(groups):
            g = padded[r, j * GROUP:(j + 1) * GROUP]
            at = slice(j * GROUP, (j + 1) * GROUP)
            if not bool(g.isfinite().all()):
                exponents[r, j] = 128  # byte 255
                values[r, at] = math.nan
                continue
            top = float(g.abs().max())
            e = -126
            while top > limit * 2.0 ** e:  # the smallest power of two that is large enough
                e += max(1, math.floor(math.log2(top / limit)) - e - 1)
            exponents[r, j] = e
            v = g / 2.0 ** e
            if form == E4M3:
                step = 2.0 ** (torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
                codes[r, at] = torch.round(v / step) * step
            else:
                codes[r, at] = torch.round(v)
            values[r, at] = codes[r, at] * 2.0 ** e
    return codes, exponents, values[:, :cols]


def embedding_backward64(dy, ids, rows, scale):
    """The gradient and the room for fp32 arithmetic in it: a row of n tokens is
    summed up to 64 + n / 128 times in a row (up to 63 tokens of a run, or parts
    of 8 tokens at least, a sixteenth of them a warp, then 16 warps), then scaled."""
    dy, ids = dy.double().reshape(-1, dy.shape[-1]), ids.reshape(-1).long()
    want = torch.zeros(rows, dy.shape[1], dtype=torch.float64)
    room = torch.zeros_like(want)
    count = torch.zeros(rows, 1, dtype=torch.float64)
    for t, i in enumerate(ids.tolist()):
        if 0 <= i < rows:
            want[i] += dy[t]
            room[i] += dy[t].abs()
            count[i] += 1
    return scale * want, (66 + count / 128) * U32 * abs(scale) * room


def power_of_two(e: torch.Tensor) -> torch.Tensor:
    """2^e in 64 bits, by the bits (-1022 <= e <= 1023)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def pack64_many(x: torch.Tensor, form: torch.dtype):
    """`pack64` for large matrices, on the device of `x`: all groups at once."""
    limit = 448.0 if form == E4M3 else 127.0
    rows, cols = x.shape
    groups = -(-cols // GROUP)
    v = torch.zeros(rows, groups * GROUP, dtype=torch.float64, device=x.device)
    v[:, :cols] = x.double()
    v = v.view(rows, groups, GROUP)
    finite = v.isfinite().all(2)
    v = torch.where(finite[..., None], v, 0.0)
    top = v.abs().amax(2)
    top = top.clamp(min=2.0 ** -160)  # (any below 2^-126)
    e = torch.frexp(top / limit).exponent.long().clamp(min=-126)  # right, or one off; an exact comparison decides
    e = torch.where(top > limit * power_of_two(e), e + 1, e)
    e = torch.where((e > -126) & (top <= limit * power_of_two(e - 1)), e - 1, e)
    v = v / power_of_two(e)[..., None]
    if form == E4M3:
        step = power_of_two(torch.frexp(v.abs().clamp(min=2.0 ** -6)).exponent.long() - 1 - 3)
        codes = torch.round(v / step) * step
    else:
        codes = torch.round(v)
    values = torch.where(finite[..., None], codes * power_of_two(e)[..., None], math.nan)
    return (codes.view(rows, -1), torch.where(finite, e, 128), values.view(rows, -1)[:, :cols])


def embedding_backward64_many(dy, ids, rows, scale):
    """`embedding_backward64` for many tokens, on the device of `dy`, with the same room."""
    dy, ids = dy.double().reshape(-1, dy.shape[-1]), ids.reshape(-1).long()
    live = (ids >= 0) & (ids < rows)
    ids, dy = ids[live], dy[live]
    want = torch.zeros(rows, dy.shape[1], dtype=torch.float64, device=dy.device)
    room, count = torch.zeros_like(want), torch.bincount(ids, minlength=rows)[:, None]
    want.index_add_(0, ids, dy)
    room.index_add_(0, ids, dy.abs())
    return scale * want, (66 + count / 128) * U32 * abs(scale) * room
