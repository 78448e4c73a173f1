"""Operators on torch tensors around the Muon step: :func:`orthogonalize`,
:func:`qk_norm_rope` and its gradients.

Each is a thin call of the C function of the same name: checks, the output and
workspace tensors, the current stream.  Tensors stay on one CUDA device; there
is no CPU path.
"""

from __future__ import annotations

import contextlib
import functools
import operator
from typing import Optional, Sequence, Tuple

import torch
from torch.autograd.function import once_differentiable

from . import binding as B
from ._current import current_device, current_stream

_DTYPES = {torch.bfloat16: B.ZERO_GRAD_BF16, torch.float32: B.ZERO_GRAD_FP32}
_CURRENT = contextlib.nullcontext()
# read-only configuration structs by their values (plain numbers: what hashes by
# identity, such as a tensor, could change its value under a kept entry)
_ns_config = functools.lru_cache(maxsize=64)(B.make_ns_config)
_qk_config = functools.lru_cache(maxsize=64)(B.zero_qk_config)
_CONTIGUOUS = torch.contiguous_format


def _on(device: torch.device):
    """Makes `device` current for a C call; the usual case costs nothing."""
    return _CURRENT if current_device() == device.index else torch.cuda.device(device)


def _stream(device: torch.device) -> int:
    return current_stream(device.index)


def _no_graph(what: str, *tensors: Optional[torch.Tensor]) -> None:
    """A result that torch.autograd would take for a constant is refused."""
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        raise ValueError(f"{what} records no gradient: detach its inputs or call it under torch.no_grad()")


def _layout(x: torch.Tensor) -> Tuple[int, int, list]:
    """Byte address, bytes of a contiguous run and the (stride, size) of the other dimensions, largest stride first."""
    size = x.element_size()
    dims = sorted(((st * size, n) for n, st in zip(x.shape, x.stride()) if n > 1), reverse=True)
    run = size
    while dims and dims[-1][0] == run:
        run *= dims.pop()[1]
    return x.data_ptr(), run, dims


def _span(run: int, dims) -> int:
    return run + sum(stride * (n - 1) for stride, n in dims)


def _apart(at: int, run: int, dims, other_run: int, other_dims) -> bool:
    """Whether a layout at 0 and another `at` bytes further (or before) share no byte; False where this cannot tell."""
    if at >= _span(run, dims) or -at >= _span(other_run, other_dims):
        return True
    if not dims or not other_dims or dims[0][0] != other_dims[0][0]:
        return False
    pitch, inner, other = dims[0][0], dims[1:], other_dims[1:]  # rows of one pitch, such as columns of one buffer
    if _span(run, inner) > pitch or _span(other_run, other) > pitch:
        return False
    at %= pitch
    return _apart(at, run, inner, other_run, other) and _apart(at - pitch, run, inner, other_run, other)


def _same(a: torch.Tensor, b: torch.Tensor) -> bool:
    return a.data_ptr() == b.data_ptr() and a.shape == b.shape and all(
        n == 1 or s == t for n, s, t in zip(a.shape, a.stride(), b.stride()))


def _check_memory(outs, ins) -> None:
    """Refuses outputs that overlap themselves, one another or an input; output
    i may be one of ins[i] itself (each element is read before it is written)."""
    for i, out in enumerate(outs):
        if out.numel() == 0:
            continue
        at, run, dims = _layout(out)
        if any(stride < _span(run, dims[d + 1:]) for d, (stride, _) in enumerate(dims)):
            raise ValueError("an output's elements overlap one another")
        others = [*outs[:i], *(t for j, some in enumerate(ins) for t in some if j != i or not _same(t, out))]
        for there, other_run, other_dims in (_layout(t) for t in others if t.numel()):
            if not _apart(there - at, run, dims, other_run, other_dims):
                raise ValueError("an output overlaps another tensor of the call")


def orthogonalize(x: torch.Tensor, *, steps: int = 5, coefficients: Sequence[float] = (3.4445, -4.7750, 2.0315),
                  eps: float = 1e-7, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Newton-Schulz orthogonalisation of a matrix or a stack of matrices.

    ``x``: bf16 or fp32, (rows, cols) or (batch, rows, cols), columns
    contiguous.  Returns (or fills ``out``, which must not overlap ``x``) bf16
    of the same shape.  Not differentiable: an ``x`` that requires a gradient is
    refused.  Products run on fp16 operands (22 bits where the smaller side is at
    most 128): with the default coefficients and up to 8 steps within 4e-3 of the
    exact result's norm, bf16's rounding included; noise outside a low rank grows
    with more steps, as it does in fp32.
    """
    _no_graph("orthogonalize", x)
    if x.dim() not in (2, 3) or x.dtype not in _DTYPES or not x.is_cuda:
        raise ValueError("x must be a bf16 or fp32 CUDA matrix or a stack of them")
    if x.size(-1) > 1 and x.stride(-1) != 1:
        raise ValueError("the columns of x must be contiguous")
    if out is None:
        out = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
    elif out.shape != x.shape or out.dtype != torch.bfloat16 or out.device != x.device or (
            out.size(-1) > 1 and out.stride(-1) != 1):
        raise ValueError("out must be a bf16 tensor of x's shape and device with contiguous columns")
    else:
        _check_memory((out,), ((), (x,)))
    batch, rows, cols = (1, *x.shape) if x.dim() == 2 else x.shape
    cfg = _ns_config(operator.index(steps), tuple(map(float, coefficients)), float(eps))
    with _on(x.device):
        need = B.zero_orthogonalize_workspace_bytes(cfg, rows, cols, batch)
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)  # 512-byte aligned
        B.zero_orthogonalize(cfg, rows, cols, batch, x.data_ptr(), _DTYPES[x.dtype],
                             x.stride(-2) if rows > 1 else max(cols, 1), x.stride(0) if batch > 1 else 0,
                             out.data_ptr(), out.stride(-2) if rows > 1 else max(cols, 1),
                             out.stride(0) if batch > 1 else 0, workspace.data_ptr(), need, _stream(x.device))
    return out


def kernel_timeouts(device: Optional[torch.device] = None) -> int:
    """Bounded waits that gave up on the device since the library was loaded:
    0, unless the hardware failed to deliver.  A call in whose course the count
    grew left part of its output unwritten.  Synchronizes."""
    device = torch.device("cuda" if device is None else device)
    with torch.cuda.device(device):
        return B.zero_kernel_timeouts()


def _heads(x: torch.Tensor) -> B.zero_heads:
    token, head, one = x.stride()
    if one != 1 and x.size(2) > 1:
        raise ValueError("the vector of a head must be contiguous")
    return B.zero_heads(x.data_ptr(), token, head)


def _check_qk(q, k, q_gain, k_gain, table, positions, eps, interleaved):
    device, dtype = q.device, q.dtype
    if q.dim() != 3 or k.dim() != 3 or dtype not in _DTYPES or not q.is_cuda:
        raise ValueError("q and k must be bf16 or fp32 CUDA tensors (tokens, heads, head_dim)")
    (tokens, q_heads, dim), (k_tokens, k_heads, k_dim) = q.shape, k.shape
    if k.dtype != dtype or k.device != device or k_tokens != tokens or k_dim != dim:
        raise ValueError("q and k must agree in type, device, tokens and head_dim")
    gain_dtype = None
    for g in (q_gain, k_gain):
        if g is None:
            continue
        if g.dtype not in _DTYPES or g.shape != (dim,) or g.device != device or not g.is_contiguous():
            raise ValueError("a gain must be a contiguous bf16 or fp32 vector of head_dim elements")
        if gain_dtype not in (None, g.dtype):
            raise ValueError("the gains must have one type")
        gain_dtype = g.dtype
    if table.dim() != 2 or table.dtype != torch.float32 or table.device != device or not table.is_contiguous():
        raise ValueError("table must be a contiguous fp32 tensor (positions, rotary_dim)")
    if positions is not None and (positions.dtype != torch.int32 or positions.shape != (tokens,)
                                  or positions.device != device or not positions.is_contiguous()):
        raise ValueError("positions must be a contiguous int32 vector with one entry per token")
    n_positions, rotary = table.shape
    return tokens, _qk_config(q_heads, k_heads, dim, rotary, 1 if interleaved else 0, _DTYPES[dtype],
                              _DTYPES[gain_dtype or torch.float32], float(eps), n_positions)


@functools.lru_cache(maxsize=256)
def _backward_workspace(q_heads: int, k_heads: int, dim: int, tokens: int, device: int) -> int:
    return B.zero_qk_backward_workspace_bytes(B.zero_qk_config(q_heads, k_heads, dim, 0, 0, 0, 0, 0.0, 0), tokens)


def _ptr(x: Optional[torch.Tensor]) -> int:
    return x.data_ptr() if x is not None else 0


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, q_gain: Optional[torch.Tensor], k_gain: Optional[torch.Tensor],
                 table: torch.Tensor, positions: Optional[torch.Tensor] = None, *, eps: float = 1e-6,
                 interleaved: bool = False, out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None
                 ) -> Tuple[torch.Tensor, torch.Tensor]:
    """RMS norm of every head of q and k (with its gain), then the rotation of
    the token's position, in one pass.

    ``q`` (tokens, heads, head_dim) and ``k`` (tokens, kv_heads, head_dim) may
    be strided views of one projection's output.  ``table`` holds per position
    the rotary_dim/2 cosines, then the sines; rotary_dim is its width.  A
    position outside the table marks padding: zeros.  ``out`` may be (q, k),
    and must not overlap them otherwise.
    Inputs that require gradients are refused: :func:`qk_norm_rope_autograd`
    records them.
    """
    _no_graph("qk_norm_rope (qk_norm_rope_autograd does)", q, k, q_gain, k_gain)
    tokens, cfg = _check_qk(q, k, q_gain, k_gain, table, positions, eps, interleaved)
    if out is None:
        out = (torch.empty_like(q, memory_format=_CONTIGUOUS), torch.empty_like(k, memory_format=_CONTIGUOUS))
    else:
        _check_like(out, (q, k))
        _check_memory(out, ((q,), (k,)))
    device = q.device
    with _on(device):
        B.zero_qk_norm_rope(cfg, tokens, _heads(q), _heads(k), _ptr(q_gain), _ptr(k_gain), table.data_ptr(),
                            _ptr(positions), _heads(out[0]), _heads(out[1]), _stream(device))
    return out


def _check_like(got, want):
    for g, w in zip(got, want):
        if g.shape != w.shape or g.dtype != w.dtype or g.device != w.device:
            raise ValueError("an output or output gradient must match its input in shape, type and device")


def qk_norm_rope_backward(dq_out: torch.Tensor, dk_out: torch.Tensor, q: torch.Tensor, k: torch.Tensor,
                          q_gain: Optional[torch.Tensor], k_gain: Optional[torch.Tensor], table: torch.Tensor,
                          positions: Optional[torch.Tensor] = None, *, eps: float = 1e-6, interleaved: bool = False,
                          out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
                          gain_out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None):
    """Gradients (dq, dk, dq_gain, dk_gain) of :func:`qk_norm_rope`'s inputs.

    ``out`` may be (dq_out, dk_out) or (q, k), and must not overlap them otherwise.
    ``gain_out``: two vectors of head_dim elements, bf16 or fp32, to write the
    gain gradients to, such as slices of a replica's flat gradient; new fp32
    vectors otherwise.  Inputs that require gradients are refused, as in
    :func:`qk_norm_rope`.
    """
    _no_graph("qk_norm_rope_backward", dq_out, dk_out, q, k, q_gain, k_gain)
    tokens, cfg = _check_qk(q, k, q_gain, k_gain, table, positions, eps, interleaved)
    _check_like((dq_out, dk_out), (q, k))
    if out is None:
        out = (torch.empty_like(q, memory_format=_CONTIGUOUS), torch.empty_like(k, memory_format=_CONTIGUOUS))
    else:
        _check_like(out, (q, k))
        _check_memory(out, ((dq_out, q), (dk_out, k)))
    device, dim = q.device, cfg.head_dim
    if gain_out is None:
        gain_out = (torch.empty(dim, dtype=torch.float32, device=device),
                    torch.empty(dim, dtype=torch.float32, device=device))
    else:
        for g in gain_out:
            if g.dtype not in _DTYPES or g.dtype != gain_out[0].dtype or g.shape != (dim,) or g.device != device \
                    or not g.is_contiguous():
                raise ValueError("gain_out must be two contiguous vectors of head_dim elements and one type")
        _check_memory(gain_out, ())
    with _on(device):
        need = max(_backward_workspace(cfg.q_heads, cfg.k_heads, dim, tokens, device.index), 16)
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
        B.zero_qk_norm_rope_backward(cfg, tokens, _heads(dq_out), _heads(dk_out), _heads(q), _heads(k),
                                     _ptr(q_gain), _ptr(k_gain), table.data_ptr(), _ptr(positions), _heads(out[0]),
                                     _heads(out[1]), gain_out[0].data_ptr(), gain_out[1].data_ptr(),
                                     _DTYPES[gain_out[0].dtype], workspace.data_ptr(), need, _stream(device))
    return (*out, *gain_out)


class _QkNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_gain, k_gain, table, positions, eps, interleaved):
        ctx.save_for_backward(q, k, q_gain, k_gain, table, positions)
        ctx.eps, ctx.interleaved = eps, interleaved
        return qk_norm_rope(q, k, q_gain, k_gain, table, positions, eps=eps, interleaved=interleaved)

    @staticmethod
    @once_differentiable  # a second derivative raises: the kernels record no graph
    def backward(ctx, dq_out, dk_out):
        q, k, q_gain, k_gain, table, positions = ctx.saved_tensors
        dq_out, dk_out = (d if d.stride(2) == 1 or d.size(2) == 1 else d.contiguous() for d in (dq_out, dk_out))
        dq, dk, dq_gain, dk_gain = qk_norm_rope_backward(dq_out, dk_out, q, k, q_gain, k_gain, table, positions,
                                                         eps=ctx.eps, interleaved=ctx.interleaved)
        return (dq, dk, dq_gain.to(q_gain.dtype) if q_gain is not None else None,
                dk_gain.to(k_gain.dtype) if k_gain is not None else None, None, None, None, None)


def qk_norm_rope_autograd(q, k, q_gain, k_gain, table, positions=None, *, eps: float = 1e-6,
                          interleaved: bool = False):
    """:func:`qk_norm_rope` that records its gradients for torch.autograd (first
    derivatives; differentiating them again raises an error)."""
    return _QkNormRope.apply(q, k, q_gain, k_gain, table, positions, eps, interleaved)
