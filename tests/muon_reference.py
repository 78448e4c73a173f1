"""Plain 64-bit forms that the tests of the Muon step and of the query / key
norm compare with, written from the formulas with torch on the CPU."""

from __future__ import annotations

import math

import torch

COEFFICIENTS = (3.4445, -4.7750, 2.0315)

# The relative error (Frobenius) that the orthogonalisation may show against
# 64 bits.  Every stored operand (Gram matrix, polynomial, iterate) is rounded
# to 11 bits: a random relative error of at most 2^-11, rms 2^-11 / sqrt(3) =
# 2.8e-4.  Three roundings per step, each passing a polynomial whose relative
# slope |s p'(s) / p(s)| stays below 4 on the way to 1, over five steps that
# add in quadrature: 2.8e-4 * sqrt(15) * 4 = 4.4e-3; the bf16 result adds 2^-9.
NS_TOL = 6e-3


def orthogonalized64(x: torch.Tensor, steps=5, coefficients=COEFFICIENTS, eps=1e-7) -> torch.Tensor:
    a, b, c = coefficients
    x = x.double()
    tall = x.shape[-2] > x.shape[-1]
    x = x.mT if tall else x
    x = x / (x.square().sum((-2, -1), keepdim=True).sqrt() + eps)
    for _ in range(steps):
        s = x @ x.mT
        x = a * x + b * (s @ x) + c * (s @ (s @ x))
    return x.mT if tall else x


def muon_scale(rows, cols, scale):
    return 0.2 * math.sqrt(max(rows, cols)) if scale == "rms" else math.sqrt(max(1.0, rows / cols))


def relative(got: torch.Tensor, want: torch.Tensor) -> float:
    got, want = got.double().cpu(), want.double().cpu()
    norm = want.norm()
    return float((got - want).norm() / norm) if norm > 0 else float((got - want).norm())


def rotation_table(n_positions: int, rotary: int, base: float = 10000.0) -> torch.Tensor:
    half = rotary // 2
    freq = torch.tensor([base ** (-i / max(half, 1)) for i in range(half)], dtype=torch.float64)
    angle = torch.arange(n_positions, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def qk64(x, gain, table, positions, eps, interleaved):
    """(tokens, heads, dim) in 64 bits; differentiable in x and gain."""
    rotary = table.shape[1]
    half = rotary // 2
    live = (positions >= 0) & (positions < table.shape[0])
    row = table.double()[torch.where(live, positions, 0).long()][:, None] if table.shape[0] else \
        torch.zeros(x.shape[0], 1, rotary, dtype=torch.float64)
    cs, sn = row[..., :half], row[..., half:]
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps)
    if gain is not None:
        y = y * gain
    if interleaved:
        one, two = y[..., 0:rotary:2], y[..., 1:rotary:2]
        turned = torch.stack([one * cs - two * sn, two * cs + one * sn], -1).flatten(-2)
    else:
        one, two = y[..., :half], y[..., half:rotary]
        turned = torch.cat([one * cs - two * sn, two * cs + one * sn], -1)
    out = torch.cat([turned, y[..., rotary:]], -1)
    return torch.where(live[:, None, None], out, torch.zeros((), dtype=torch.float64))
