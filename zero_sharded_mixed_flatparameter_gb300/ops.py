"""Operators on torch tensors around the optimizer step: :func:`orthogonalize`,
:func:`qk_norm_rope`, :func:`layer_norm` and :func:`embedding` with their
gradients, and activations kept in 8 bits (:func:`pack_activations`).

Each is a thin call of the C function of the same name: checks, the output and
workspace tensors, the current stream.  Tensors stay on one CUDA device; there
is no CPU path.

The functions without autograd can be captured into CUDA graphs as they are.  Of
the ``*_autograd`` ones, capture the forward and the backward pass together, while
no graph of an earlier forward pass over the same leaves is alive: torch would
make the capture wait for that one's stream.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
import operator
from typing import Optional, Sequence, Tuple, Union

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


@functools.lru_cache(maxsize=64)
def _norm_config(*values):
    return ctypes.byref(B.zero_norm_config(*values))


@functools.lru_cache(maxsize=64)
def _embedding_config(*values):
    return ctypes.byref(B.zero_embedding_config(*values))


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


def _no_leaf(*outs: Optional[torch.Tensor]) -> None:
    """An output that requires a gradient is refused: torch.autograd would not learn of what is written."""
    for t in outs:
        if t is not None and t.requires_grad and torch.is_grad_enabled():
            raise ValueError("an output requires a gradient: detach it or call under torch.no_grad()")


# Tells torch.autograd that the kernels wrote to tensors of the caller's, so that a
# backward pass that saved one of them raises instead of reading what is there now.
_written = torch.autograd.graph.increment_version


def _layout(x: torch.Tensor) -> Tuple[int, int, Sequence]:
    """Byte address, bytes of a contiguous run and the (stride, size) of the other dimensions, largest stride first."""
    size = x.element_size()
    if x.is_contiguous():
        return x.data_ptr(), x.numel() * size, ()
    dims = sorted(((st * size, n) for n, st in zip(x.shape, x.stride()) if n > 1), reverse=True)
    run = size
    while dims and dims[-1][0] == run:
        run *= dims.pop()[1]
    return x.data_ptr(), run, dims


def _span(run: int, dims) -> int:
    return run + sum(stride * (n - 1) for stride, n in dims) if dims else run


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


def _given(*tensors: Optional[torch.Tensor]) -> list:
    return [t for t in tensors if t is not None]


def _check_memory(outs, ins) -> None:
    """Refuses outputs that overlap themselves, one another or an input; output
    i may be one of ins[i] itself (each element is read before it is written)."""
    for i, out in enumerate(outs):
        if out.numel() == 0:
            continue
        at, run, dims = _layout(out)
        if dims and any(stride < _span(run, dims[d + 1:]) for d, (stride, _) in enumerate(dims)):
            raise ValueError("an output's elements overlap one another")
        end = at + _span(run, dims)
        for j, some in enumerate((outs[:i], *ins), -1):
            for t in some:
                there = t.data_ptr()
                if there >= end or t.numel() == 0:  # the usual case: memory of its own
                    continue
                _, other_run, other_dims = _layout(t)
                if there + _span(other_run, other_dims) <= at or j == i and _same(t, out):
                    continue
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
        _no_leaf(out)
        _check_memory((out,), ((), (x,)))
        _written(out)
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
    and must not overlap an input otherwise.
    Inputs that require gradients are refused: :func:`qk_norm_rope_autograd`
    records them.
    """
    _no_graph("qk_norm_rope (qk_norm_rope_autograd does)", q, k, q_gain, k_gain)
    tokens, cfg = _check_qk(q, k, q_gain, k_gain, table, positions, eps, interleaved)
    if out is None:
        out = (torch.empty_like(q, memory_format=_CONTIGUOUS), torch.empty_like(k, memory_format=_CONTIGUOUS))
    else:
        _no_leaf(*out)
        _check_like(out, (q, k))
        _check_memory(out, ((q,), (k,), _given(q_gain, k_gain, table, positions)))
        _written(out)
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

    ``out`` may be (dq_out, dk_out) or (q, k), and must not overlap an input otherwise.
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
        _no_leaf(*out)
        _check_like(out, (q, k))
        _check_memory(out, ((dq_out, q), (dk_out, k), _given(q_gain, k_gain, table, positions)))
        _written(out)
    device, dim = q.device, cfg.head_dim
    if gain_out is None:
        gain_out = (torch.empty(dim, dtype=torch.float32, device=device),
                    torch.empty(dim, dtype=torch.float32, device=device))
    else:
        _no_leaf(*gain_out)
        for g in gain_out:
            if g.dtype not in _DTYPES or g.dtype != gain_out[0].dtype or g.shape != (dim,) or g.device != device \
                    or not g.is_contiguous():
                raise ValueError("gain_out must be two contiguous vectors of head_dim elements and one type")
        _check_memory(gain_out, ((), (), out))
        _written(gain_out)
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


# ---- rows of activations -------------------------------------------------------
# Called for every layer of a step, or for every new token: checks stand together
# and the usual layouts first, since the host's share of a small call is larger
# than the kernel's.
_FORMATS = {torch.float8_e4m3fn: B.ZERO_PACK_E4M3, torch.int8: B.ZERO_PACK_INT8}
_GROUP = 32  # columns that share a scale
_grad_enabled = torch.is_grad_enabled


def _call(function, device: torch.device, *args) -> None:
    """A C function on the device's current stream."""
    index = device.index
    if current_device() == index:
        status = function(*args, current_stream(index))
    else:
        with torch.cuda.device(device):
            status = function(*args, current_stream(index))
    if status:
        B._check(status)


def _matrix(x: torch.Tensor, what: str, copy: bool = True) -> torch.Tensor:
    """`x`, which has columns, as a matrix of its last dimension's rows; a copy where its strides allow no such view
    (refused unless `copy`)."""
    if x.dim() != 2:
        x = x.detach()
        if x.numel() == 0:
            x = x.new_empty((x.shape[:-1].numel(), x.size(-1)))
        elif copy:
            x = x.reshape(-1, x.size(-1))
        else:
            try:
                x = x.view(-1, x.size(-1))
            except RuntimeError:
                raise ValueError(f"the rows of {what} must have one stride") from None
    if x.stride(1) != 1 and x.size(1) > 1:
        raise ValueError(f"the columns of {what} must be contiguous")
    return x


def _new_like(x: torch.Tensor) -> torch.Tensor:
    """A contiguous tensor of x's shape, type and device."""
    return torch.empty_like(x) if x.is_contiguous() else torch.empty_like(x, memory_format=_CONTIGUOUS)


def _check_rows(x: torch.Tensor, what: str) -> int:
    """The type of a tensor of rows."""
    dtype = _DTYPES.get(x.dtype)
    if dtype is None or not x.is_cuda:
        raise ValueError(f"{what} must be a bf16 or fp32 CUDA tensor")
    if x.dim() == 0 or x.size(-1) == 0:
        raise ValueError(f"{what} must have columns")
    return dtype


def _check_vector(v: torch.Tensor, cols: int, device: torch.device, kind: Optional[int]) -> int:
    """The type of a vector, which must be `kind` if that is given."""
    its = _DTYPES.get(v.dtype)
    if its is None or kind not in (None, its) or v.device != device or v.dim() != 1 or v.numel() != cols or \
            not v.is_contiguous():
        raise ValueError("weight, bias and their gradients must be contiguous vectors of one entry per column, those of "
                         "one call of one type (bf16 or fp32)")
    return its


class PackedActivations:
    """A tensor in 8 bits, as :func:`pack_activations` returns it.

    ``data``: the bytes, codes of 32 columns a group, then a scale a group;
    ``form``: torch.float8_e4m3fn or torch.int8; ``shape`` and ``dtype`` of what
    was packed.  ``codes`` (rows, 32 * groups) and ``scales`` (rows, groups; the
    power of two plus 127) are views of ``data``.
    """
    __slots__ = ("data", "form", "shape", "dtype", "rows", "cols", "_struct")

    def __init__(self, data: torch.Tensor, form: torch.dtype, shape: Sequence[int], dtype: torch.dtype):
        shape = torch.Size(shape)
        if form not in _FORMATS or dtype not in _DTYPES or len(shape) == 0 or min(shape) < 0 or shape[-1] == 0:
            raise ValueError("packed activations are e4m3 or int8 codes of a bf16 or fp32 tensor with columns")
        rows, cols = shape[:-1].numel(), shape[-1]
        if data.dtype != torch.uint8 or not data.is_cuda or not data.is_contiguous() or \
                data.shape != (rows * -(-cols // _GROUP) * (_GROUP + 1),):
            raise ValueError("data must be a contiguous CUDA vector of the codes' and scales' bytes")
        self._set(data, form, shape, dtype, rows, cols)

    def _set(self, data, form, shape, dtype, rows, cols):
        self.data, self.form, self.shape, self.dtype, self.rows, self.cols = data, form, shape, dtype, rows, cols
        at = data.data_ptr()
        self._struct = ctypes.byref(B.zero_packed(at, at + rows * -(-cols // _GROUP) * _GROUP, _FORMATS[form]))
        return self

    @property
    def codes(self) -> torch.Tensor:
        groups = -(-self.cols // _GROUP)
        return self.data[:self.rows * groups * _GROUP].view(self.form).view(self.rows, groups * _GROUP)

    @property
    def scales(self) -> torch.Tensor:
        groups = -(-self.cols // _GROUP)
        return self.data[self.rows * groups * _GROUP:].view(self.rows, groups)


def _new_packed(rows: int, cols: int, shape, dtype: torch.dtype, form: torch.dtype, device) -> PackedActivations:
    if form not in _FORMATS:
        raise ValueError("activations are packed to torch.float8_e4m3fn or torch.int8")
    data = torch.empty(rows * -(-cols // _GROUP) * (_GROUP + 1), dtype=torch.uint8, device=device)
    return PackedActivations.__new__(PackedActivations)._set(data, form, shape, dtype, rows, cols)


def pack_activations(x: torch.Tensor, dtype: torch.dtype = torch.float8_e4m3fn, *,
                     out: Optional[PackedActivations] = None) -> PackedActivations:
    """``x`` (bf16 or fp32, any shape, columns contiguous) in 8 bits, with a
    power-of-two scale for every 32 columns of a row.

    ``dtype``: torch.float8_e4m3fn (each entry within 2^-4 of itself or, where it is
    smaller than 2^-6 of the scale, within 2^-10 of the scale) or torch.int8 (within
    half a scale).  But for the smallest scale, 2^-126, the group's largest is above
    224 or 63.5 scales: whole numbers are within 1/127 of it.  A group with an inf or NaN reads as NaN; finite entries that round up
    to 2^128 read as inf.  ``out``: an earlier result of the same shape and types to
    write to.  What ``x`` requires a gradient for is not recorded: this keeps a
    tensor for the backward pass, as saving it would.
    """
    kind = _check_rows(x, "x")
    m, device = _matrix(x, "x"), x.device
    rows, cols = m.shape
    if out is None:
        out = _new_packed(rows, cols, x.shape, x.dtype, dtype, device)
    else:
        if out.shape != x.shape or out.dtype != x.dtype or out.form != dtype or out.data.device != device:
            raise ValueError("out must have x's shape, type and device, and codes of dtype")
        _check_memory((out.data,), ((), (m,)))
        _written(out.data)
    _call(B.load().zero_pack_activations, device, rows, cols, m.data_ptr(), kind, m.stride(0), out._struct)
    return out


def unpack_activations(packed: PackedActivations, dtype: Optional[torch.dtype] = None, *,
                       out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The values that ``packed`` stands for, in the type of what was packed or
    ``dtype`` (bf16 or fp32; both hold them exactly, but for bf16 subnormals and
    2^128, which becomes inf)."""
    device = packed.data.device
    if out is None:
        kind = _DTYPES.get(dtype or packed.dtype)
        if kind is None:
            raise ValueError("dtype must be bf16 or fp32")
        out = torch.empty(packed.shape, dtype=dtype or packed.dtype, device=device)
        at, stride = out.data_ptr(), packed.cols
    else:
        _no_leaf(out)
        kind = _DTYPES.get(out.dtype)
        if kind is None or out.shape != packed.shape or out.device != device or dtype not in (None, out.dtype):
            raise ValueError("out must be a bf16 or fp32 tensor of packed's shape and device")
        m = _matrix(out, "out", copy=False)
        _check_memory((m,), ((), (packed.data,)))
        _written(out)
        at, stride = m.data_ptr(), m.stride(0)
    _call(B.load().zero_unpack_activations, device, packed.rows, packed.cols, packed._struct, at, kind, stride)
    return out


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None, *,
               eps: float = 1e-5, center: bool = True, pack: Optional[torch.dtype] = None,
               out: Optional[torch.Tensor] = None):
    """Layer norm over the last dimension, or, with ``center=False``, the norm
    without the mean (RMS norm).

    ``x``: bf16 or fp32, any leading dimensions, columns contiguous; ``weight``
    and ``bias`` bf16 or fp32 vectors of one type.  Returns y and the rows'
    statistics (fp32, rows x 2: mean and 1 / deviation), which the backward pass
    reads; with ``pack`` (torch.float8_e4m3fn or torch.int8) also ``x`` in 8 bits
    (:class:`PackedActivations`), written in the same pass, which it can read in
    place of ``x``.  ``out`` may be ``x``, and must not overlap an input otherwise.
    Inputs that require gradients are refused: :func:`layer_norm_autograd`
    records them.
    """
    if _grad_enabled() and (x.requires_grad or weight is not None and weight.requires_grad
                            or bias is not None and bias.requires_grad):
        _no_graph("layer_norm (layer_norm_autograd does)", x, weight, bias)
    kind, device = _check_rows(x, "x"), x.device
    m = _matrix(x, "x")
    rows, cols = m.shape
    vector_kind = None if weight is None else _check_vector(weight, cols, device, None)
    if bias is not None:
        vector_kind = _check_vector(bias, cols, device, vector_kind)
    if out is None:
        out = _new_like(x)
        y, y_stride = out, cols
    else:
        _no_leaf(out)
        _check_like((out,), (x,))
        y = _matrix(out, "out", copy=False)
        y_stride = y.stride(0)
        _check_memory((y,), ((m,), _given(weight, bias)))
        _written(out)
    stats = torch.empty((rows, 2), dtype=torch.float32, device=device)
    packed = None if pack is None else _new_packed(rows, cols, x.shape, x.dtype, pack, device)
    cfg = _norm_config(cols, 1 if center else 0, kind, vector_kind or 0, float(eps))
    _call(B.load().zero_layer_norm, device, cfg, rows, m.data_ptr(), m.stride(0),
          0 if weight is None else weight.data_ptr(), 0 if bias is None else bias.data_ptr(), y.data_ptr(), y_stride,
          stats.data_ptr(), None if packed is None else packed._struct)
    return (out, stats) if packed is None else (out, stats, packed)


@functools.lru_cache(maxsize=256)
def _norm_workspace(cols: int, rows: int, device: int) -> int:
    with torch.cuda.device(device):
        return B.zero_layer_norm_backward_workspace_bytes(B.zero_norm_config(cols, 1, 0, 0, 0.0), rows)


def layer_norm_backward(dy: torch.Tensor, x: Union[torch.Tensor, PackedActivations], weight: Optional[torch.Tensor],
                        stats: torch.Tensor, *, center: bool = True, bias: bool = True,
                        out: Optional[torch.Tensor] = None, weight_out: Optional[torch.Tensor] = None,
                        bias_out: Optional[torch.Tensor] = None):
    """Gradients (dx, dweight, dbias) of :func:`layer_norm`'s inputs.

    ``x``: the forward input, or its 8-bit form, whose values then take the
    input's place.  ``stats``, ``center``: as in the forward pass; dweight is None
    without a weight, dbias with ``bias=False``.  ``out`` may be ``dy`` or ``x``,
    and must not overlap an input otherwise.  ``weight_out``, ``bias_out``: vectors of
    one type, bf16 or fp32, to write those gradients to, such as slices of a
    replica's flat gradient; new fp32 vectors otherwise.  Inputs that require
    gradients are refused.
    """
    kept = isinstance(x, PackedActivations)
    if _grad_enabled() and (dy.requires_grad or not kept and x.requires_grad
                            or weight is not None and weight.requires_grad):
        _no_graph("layer_norm_backward", dy, None if kept else x, weight)
    kind, device = _check_rows(dy, "dy"), dy.device
    g = _matrix(dy, "dy")
    rows, cols = g.shape
    vector_kind = None if weight is None else _check_vector(weight, cols, device, None)
    if kept:
        if x.shape != dy.shape or x.data.device != device:
            raise ValueError("x and dy must agree in shape and device")
        m = None
    else:
        _check_like((dy,), (x,))
        m = _matrix(x, "x")
    if stats.dtype != torch.float32 or stats.shape != (rows, 2) or stats.device != device or not stats.is_contiguous():
        raise ValueError("stats must be the contiguous fp32 tensor (rows, 2) of the forward pass")
    if out is None:
        out = _new_like(dy)
        d, d_stride = out, cols
    else:
        _no_leaf(out)
        _check_like((out,), (dy,))
        d = _matrix(out, "out", copy=False)
        d_stride = d.stride(0)
        others = _given(stats, weight)
        _check_memory((d,), ((g,), [*others, x.data]) if kept else ((g, m), others))
        _written(out)
    given = None
    if weight_out is not None or bias_out is not None:
        _no_leaf(weight_out, bias_out)
        for v in (weight_out, bias_out):
            given = given if v is None else _check_vector(v, cols, device, given)
        if bias_out is not None and not bias:
            raise ValueError("bias_out without a bias")
        mine = _given(weight_out, bias_out)
        _check_memory(mine, ((), (), (g, d, x.data if kept else m)))
        _written(mine)
    vectors = torch.bfloat16 if given == B.ZERO_GRAD_BF16 else torch.float32
    if weight is not None and weight_out is None:
        weight_out = torch.empty(cols, dtype=vectors, device=device)
    if bias and bias_out is None:
        bias_out = torch.empty(cols, dtype=vectors, device=device)
    need = 0 if weight_out is None and bias_out is None else _norm_workspace(cols, rows, device.index)
    cfg = _norm_config(cols, 1 if center else 0, kind, vector_kind or 0, 0.0)
    workspace = torch.empty(need or 16, dtype=torch.uint8, device=device)
    _call(B.load().zero_layer_norm_backward, device, cfg, rows, g.data_ptr(), g.stride(0),
          0 if kept else m.data_ptr(), 0 if kept else m.stride(0), x._struct if kept else None,
          0 if weight is None else weight.data_ptr(), stats.data_ptr(), d.data_ptr(), d_stride, _ptr(weight_out),
          _ptr(bias_out), _DTYPES[vectors], workspace.data_ptr(), need)
    return out, weight_out, bias_out


def _with_rows(d: torch.Tensor) -> torch.Tensor:
    """A gradient as the kernels take it (autograd hands over broadcast ones)."""
    return d if d.dim() and (d.stride(-1) == 1 or d.size(-1) == 1) else d.contiguous()


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, center, pack):
        x = _with_rows(x)
        y, stats, *packed = layer_norm(x, weight, bias, eps=eps, center=center, pack=pack)
        ctx.center, ctx.packed = center, None
        if packed:
            ctx.packed = pack, x.shape, x.dtype
            x = packed[0].data
        ctx.save_for_backward(x, weight, bias, stats)
        return y

    @staticmethod
    @once_differentiable  # a second derivative raises: the kernels record no graph
    def backward(ctx, dy):
        x, weight, bias, stats = ctx.saved_tensors
        if ctx.packed:
            x = PackedActivations(x, *ctx.packed)
        dx, dweight, dbias = layer_norm_backward(_with_rows(dy), x, weight, stats, center=ctx.center,
                                                 bias=bias is not None)
        return (dx, dweight.to(weight.dtype) if weight is not None else None,
                dbias.to(bias.dtype) if bias is not None else None, None, None, None)


def layer_norm_autograd(x, weight=None, bias=None, *, eps: float = 1e-5, center: bool = True,
                        pack: Optional[torch.dtype] = None) -> torch.Tensor:
    """:func:`layer_norm`'s y, recording its gradients for torch.autograd (first
    derivatives; differentiating them again raises an error).  With ``pack`` the
    8-bit form of ``x`` is kept for the backward pass in place of ``x``: a half or
    a quarter of the memory, for gradients of weight and ``x`` through the rounded
    entries."""
    return _LayerNorm.apply(x, weight, bias, eps, center, pack)


_ID_BYTES = {torch.int32: 4, torch.int64: 8}


def _check_ids(ids: torch.Tensor, device: torch.device) -> Tuple[torch.Tensor, int]:
    """`ids` contiguous, and the bytes of one."""
    size = _ID_BYTES.get(ids.dtype)
    if size is None or ids.device != device:
        raise ValueError("ids must be an int32 or int64 tensor on the device of the others")
    return (ids if ids.is_contiguous() else ids.contiguous()), size


def embedding(ids: torch.Tensor, table: torch.Tensor, *, scale: float = 1.0,
              out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``scale`` times the rows ``ids`` of ``table``, rounded once; zeros where an
    id is outside the table (padding).

    ``ids``: int32 or int64, any shape; ``table`` (rows, dim) bf16 or fp32 with
    contiguous columns, such as a slice of the gathered unit buffer.  Returns (or
    fills ``out``) ids.shape + (dim,).  A ``table`` that requires a gradient is
    refused: :func:`embedding_autograd` records it.
    """
    if table.requires_grad:
        _no_graph("embedding (embedding_autograd does)", table)
    kind, device = _check_rows(table, "table"), table.device
    if table.dim() != 2 or (table.stride(1) != 1 and table.size(1) > 1):
        raise ValueError("table must be a matrix with contiguous columns")
    rows, dim = table.shape
    ids, size = _check_ids(ids, device)
    if out is None:
        out = torch.empty((*ids.shape, dim), dtype=table.dtype, device=device)
        at, stride = out.data_ptr(), dim
    else:
        _no_leaf(out)
        if out.shape != (*ids.shape, dim) or out.dtype != table.dtype or out.device != device:
            raise ValueError("out must have the shape of ids and dim, and table's type and device")
        y = _matrix(out, "out", copy=False)
        at, stride = y.data_ptr(), y.stride(0)
        _check_memory((y,), ((), (table, ids)))
        _written(out)
    cfg = _embedding_config(rows, dim, kind, size, float(scale))
    _call(B.load().zero_embedding, device, cfg, ids.numel(), ids.data_ptr(), table.data_ptr(), table.stride(0), at, stride)
    return out


@functools.lru_cache(maxsize=256)
def _embedding_workspace(rows: int, dim: int, tokens: int) -> int:
    return B.zero_embedding_backward_workspace_bytes(B.zero_embedding_config(rows, dim, 0, 4, 1.0), tokens)


def embedding_backward(dy: torch.Tensor, ids: torch.Tensor, rows: int, *, scale: float = 1.0,
                       out: Optional[torch.Tensor] = None, accumulate: bool = False) -> torch.Tensor:
    """Gradient (rows, dim) of :func:`embedding`'s table from that of its result:
    every row ``scale`` times the sum over its tokens, in fp32 and in a fixed order.

    ``out``: a bf16 or fp32 matrix to write it to, such as a slice of a replica's
    flat gradient; a new one of ``dy``'s type otherwise.  Rows without tokens are
    zeroed; with ``accumulate`` the sums are added to ``out`` instead, and those
    rows stay as they are.
    """
    if dy.requires_grad:
        _no_graph("embedding_backward", dy)
    kind, device, dim, rows = _check_rows(dy, "dy"), dy.device, dy.size(-1), operator.index(rows)
    ids, size = _check_ids(ids, device)
    if dy.shape[:-1] != ids.shape:
        raise ValueError("dy must have the shape of ids and one more dimension")
    g = _matrix(dy, "dy")
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs an out to add to")
        out, out_kind = torch.empty((rows, dim), dtype=dy.dtype, device=device), kind
    else:
        _no_leaf(out)
        out_kind = _DTYPES.get(out.dtype)
        if out_kind is None or out.shape != (rows, dim) or out.device != device or (out.stride(1) != 1 and dim > 1):
            raise ValueError("out must be a bf16 or fp32 matrix (rows, dim) with contiguous columns")
        _check_memory((out,), ((), (g, ids)))
        _written(out)
    tokens = ids.numel()
    cfg, need = _embedding_config(rows, dim, kind, size, float(scale)), _embedding_workspace(rows, dim, tokens)
    workspace = torch.empty(need, dtype=torch.uint8, device=device)
    _call(B.load().zero_embedding_backward, device, cfg, tokens, ids.data_ptr(), g.data_ptr(), g.stride(0),
          out.data_ptr(), out_kind, out.stride(0), 1 if accumulate else 0, workspace.data_ptr(), need)
    return out


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, table, scale):
        ctx.save_for_backward(ids)
        ctx.rows, ctx.scale = table.size(0), scale
        return embedding(ids, table, scale=scale)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        return None, embedding_backward(_with_rows(dy), ctx.saved_tensors[0], ctx.rows, scale=ctx.scale), None


def embedding_autograd(ids, table, *, scale: float = 1.0) -> torch.Tensor:
    """:func:`embedding` that records the table's gradient for torch.autograd
    (first derivatives; differentiating it again raises an error)."""
    return _Embedding.apply(ids, table, scale)
