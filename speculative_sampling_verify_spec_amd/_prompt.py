"""Binding of whole prompts (argument marshalling only): prompt_attention,
prompt_weights.
Checks shapes and dtypes, allocates outputs with torch and passes device
pointers plus torch's current stream of the tensors' device."""
from __future__ import annotations

from typing import Optional

from . import _kv
from ._kv import KV_DIMS, _bind_torch, _call, _dtype_code, _forward_only
from ._lib import load


def _row(name: str, t, heads: int, dim: int) -> int:
    """Elements between the token rows of t [T, heads, dim]: heads and channels
    contiguous (a slice of a fused projection's rows will do)."""
    row, head, channel = t.stride()
    if t.shape[0] <= 1 or t.is_contiguous():
        row = heads * dim
    if (channel != 1 or (heads > 1 and head != dim)) and t.numel():
        raise ValueError(f"{name}: heads and channels must be contiguous")
    if row < heads * dim:
        raise ValueError(f"{name}: tokens must be evenly spaced and must not overlap")
    return row


def _packed(q, k, starts):
    """Checks of packed prompts: (T, Hq, dim, heads, sequences, q's stride, k's stride, dtype's code)."""
    device = q.device
    if device.type != "cuda":
        raise ValueError("q must be on a GPU")
    if q.dim() != 3:
        raise ValueError("q must be [T, Hq, dim]")
    T, Hq, dim = q.shape
    if dim not in KV_DIMS:
        raise ValueError(f"dim must be one of {KV_DIMS}, got {dim}")
    code = _dtype_code(q.dtype)
    if k.dim() != 3 or k.shape[0] != T or k.shape[2] != dim or k.device != device or k.dtype is not q.dtype:
        raise ValueError(f"k must be [{T}, heads, {dim}], with q's dtype and on q's device")
    heads = k.shape[1]
    if Hq < 1 or heads < 1 or Hq % heads:
        raise ValueError(f"q's {Hq} heads must be a multiple of k's {heads}")
    if starts.dtype is not _kv.torch.int32 or starts.dim() != 1 or starts.shape[0] < 2 or starts.device != device or \
            not starts.is_contiguous():
        raise ValueError("starts must be a contiguous int32 [B + 1] tensor on q's device")
    return T, Hq, dim, heads, starts.shape[0] - 1, _row("q", q, Hq, dim), _row("k", k, heads, dim), code


def prompt_attention(q, k, v, starts, *, scale: Optional[float] = None, return_lse: bool = False):
    """Causal attention of whole prompts, packed (spec_prompt_attention).

    q [T, Hq, dim], k and v [T, heads, dim] (bf16 or fp32; slices of a fused
    projection's rows will do; k and v with the same strides), Hq a multiple of
    heads; starts [B + 1] int32, ascending: sequence b has the rows starts[b] ..
    starts[b+1]-1.  scale defaults to dim ** -0.5.  Returns out [T, Hq, dim]
    and, when asked, lse [T, Hq] float32; rows of no sequence are 0 and
    -infinity.  Forward only: a backward pass through the results raises
    NotImplementedError."""
    _bind_torch()
    T, Hq, dim, heads, B, q_row, kv_row, code = _packed(q, k, starts)
    if v.shape != k.shape or v.device != q.device or v.dtype is not q.dtype or _row("v", v, heads, dim) != kv_row:
        raise ValueError("v must have k's shape, dtype, strides and device")
    torch = _kv.torch
    out = torch.empty((T, Hq, dim), dtype=q.dtype, device=q.device)
    lse = torch.empty((T, Hq), dtype=torch.float32, device=q.device) if return_lse else None
    if T:
        _call(q.device, load().spec_prompt_attention, q.data_ptr(), q_row, k.data_ptr(), v.data_ptr(), kv_row,
              starts.data_ptr(), dim ** -0.5 if scale is None else float(scale), B, T, heads, Hq, dim,
              out.data_ptr(), lse.data_ptr() if return_lse else None, code)
    results = _forward_only((out, lse) if return_lse else (out,), (q, k, v), "prompt_attention")
    return results if return_lse else results[0]


def prompt_weights(q, k, lse, starts, capacity: int, *, scale: Optional[float] = None):
    """The attention weight that the tokens of packed prompts gather from the
    prompts themselves (spec_prompt_weights).

    q, k, starts and scale as for prompt_attention, lse [T, Hq] float32 as it
    returns it (infinite: a query that weighs nothing).  Returns weights [B,
    heads, capacity] float32: by token of the sequence, the sum of e^(score -
    lse) over the queries that see it and the query heads of its head; 0 behind
    the sequence (tokens at and behind capacity are left out).  Without
    gradients."""
    _bind_torch()
    T, Hq, dim, heads, B, q_row, kv_row, code = _packed(q, k, starts)
    if lse.dtype is not _kv.torch.float32 or lse.shape != (T, Hq) or lse.device != q.device or not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous float32 [{T}, {Hq}] tensor on q's device")
    if capacity < 1:
        raise ValueError("capacity must be at least 1")
    weights = _kv.torch.empty((B, heads, capacity), dtype=_kv.torch.float32, device=q.device)
    if not T:
        return weights.zero_()
    _call(q.device, load().spec_prompt_weights, q.data_ptr(), q_row, k.data_ptr(), kv_row, lse.data_ptr(),
          starts.data_ptr(), dim ** -0.5 if scale is None else float(scale), B, T, heads, Hq, dim,
          weights.data_ptr(), capacity, code)
    return weights
