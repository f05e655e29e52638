"""Binding of the 8-bit paged cache (argument marshalling only): KVCache,
kv_append, kv_read, kv_attention, kv_weights, kv_evict.  Checks shapes and dtypes, allocates outputs
and workspaces with torch and passes device pointers plus torch's current
stream of the tensors' device."""
from __future__ import annotations

import struct
from typing import Optional

from ._lib import SPECV_BF16, SPECV_F32, SpecVerifyError, _ptr, load, strerror

SPECV_E4M3, SPECV_I8 = 0, 1
KV_PAGE_SIZES = (16, 32, 64, 128)
KV_DIMS = (64, 96, 128, 256)


torch = None  # bound by the first cache or prompt: the package imports without it
_ForwardOnly = None


def _bind_torch() -> None:
    global torch, _ForwardOnly
    if torch is None:
        import torch as t

        class ForwardOnly(t.autograd.Function):
            """Hands results through; a backward pass that reaches them is an error."""

            @staticmethod
            def forward(ctx, name, n, *tensors):
                ctx.name = name
                ctx.mark_dirty(*tensors[:n])  # the tensors themselves, not views of them, which refuse in-place work
                return tensors[:n]

            @staticmethod
            def backward(ctx, *grads):
                raise NotImplementedError(f"{ctx.name} is forward only: it has no gradients")

        torch, _ForwardOnly = t, ForwardOnly


def _forward_only(results, inputs, name="kv_attention"):
    """The results; where autograd follows the inputs, tied to them, so that
    gradients are refused and not left out."""
    if torch.is_grad_enabled():
        inputs = [t for t in inputs if t is not None and t.requires_grad]
        if inputs:
            return _ForwardOnly.apply(name, len(results), *results, *inputs)
    return results


class KVCache:
    """The pages and scales of an 8-bit cache.

    k_pages [num_pages, heads, page_size, dim] and v_pages [num_pages, heads,
    dim, page_size] (transposed) in torch.float8_e4m3fn or torch.int8,
    k_scales and v_scales [num_pages, heads] float32, all contiguous on one
    device.  KVCache.empty() allocates them."""

    __slots__ = ("_k", "_v", "_ks", "_vs", "_device", "_type", "_pages", "_heads", "_page", "_dim")

    def __init__(self, k_pages, v_pages, k_scales, v_scales):
        _bind_torch()
        if k_pages.dim() != 4:
            raise ValueError("k_pages must be [num_pages, heads, page_size, dim]")
        n, h, p, d = k_pages.shape
        if k_pages.dtype not in (torch.float8_e4m3fn, torch.int8) or v_pages.dtype != k_pages.dtype:
            raise TypeError(f"pages must both be torch.float8_e4m3fn or torch.int8, got {k_pages.dtype} and "
                            f"{v_pages.dtype}")
        if p not in KV_PAGE_SIZES or d not in KV_DIMS:
            raise ValueError(f"page size must be one of {KV_PAGE_SIZES} and dim one of {KV_DIMS}, got {p} and {d}")
        if tuple(v_pages.shape) != (n, h, d, p):
            raise ValueError("v_pages must be [num_pages, heads, dim, page_size]")
        for t in (k_scales, v_scales):
            if t.dtype != torch.float32 or tuple(t.shape) != (n, h):
                raise ValueError("scales must be float32 [num_pages, heads]")
        for t in (k_pages, v_pages, k_scales, v_scales):
            if t.device != k_pages.device or not t.is_contiguous():
                raise ValueError("pages and scales must be contiguous tensors on the same device")
        self._k, self._v, self._ks, self._vs = k_pages, v_pages, k_scales, v_scales
        self._device = k_pages.device
        self._pages, self._heads, self._page, self._dim = n, h, p, d
        self._type = SPECV_I8 if k_pages.dtype == torch.int8 else SPECV_E4M3

    @classmethod
    def empty(cls, num_pages: int, page_size: int, heads: int, dim: int, dtype=None, device="cuda") -> "KVCache":
        """A cache of num_pages pages (dtype: torch.float8_e4m3fn, the default, or torch.int8)."""
        _bind_torch()
        dtype = torch.float8_e4m3fn if dtype is None else dtype
        return cls(torch.empty((num_pages, heads, page_size, dim), dtype=dtype, device=device),
                   torch.empty((num_pages, heads, dim, page_size), dtype=dtype, device=device),
                   torch.empty((num_pages, heads), dtype=torch.float32, device=device),
                   torch.empty((num_pages, heads), dtype=torch.float32, device=device))

    @property
    def k_pages(self):
        return self._k

    @property
    def v_pages(self):
        return self._v

    @property
    def k_scales(self):
        return self._ks

    @property
    def v_scales(self):
        return self._vs

    @property
    def device(self):
        return self._device

    @property
    def page_size(self) -> int:
        return self._page

    @property
    def heads(self) -> int:
        return self._heads

    @property
    def dim(self) -> int:
        return self._dim


_pack = struct.Struct("@5P6i").pack  # specv_kv_t, read by the library during the call


def _descriptor(cache: KVCache, table_ptr: int, max_pages: int) -> bytes:
    return _pack(cache._k.data_ptr(), cache._v.data_ptr(), cache._ks.data_ptr(), cache._vs.data_ptr(), table_ptr,
                 cache._pages, max_pages, cache._page, cache._heads, cache._dim, cache._type)


def _dtype_code(dtype) -> int:
    if dtype is torch.bfloat16:
        return SPECV_BF16
    if dtype is torch.float32:
        return SPECV_F32
    raise TypeError(f"queries, keys and values must be torch.bfloat16 or torch.float32, got {dtype}")


def _check_table(cache: KVCache, page_table) -> None:
    if cache._device.type != "cuda":
        raise ValueError("the cache must be on a GPU")
    if page_table.dtype is not torch.int32 or page_table.dim() != 2 or page_table.device != cache._device or \
            not page_table.is_contiguous():
        raise ValueError("page_table must be a contiguous int32 [B, max_pages] tensor on the cache's device")


def _check_ints(cache: KVCache, shape, name: str, t) -> None:
    if t.dtype is not torch.int32 or t.shape != shape or t.device != cache._device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 {list(shape)} tensor on the cache's device")


def _token_stride(name: str, t, heads: int, dim: int) -> int:
    """Elements between the token rows of t [B, N, heads, dim]: heads and
    channels contiguous, one stride for all tokens (a slice of a fused
    projection's rows will do)."""
    if t.is_contiguous():
        return heads * dim
    B, N, _, _ = t.shape
    sb, sn, sh, sd = t.stride()
    if sd != 1 or (heads > 1 and sh != dim):
        raise ValueError(f"{name}: heads and channels must be contiguous")
    row = sn if N > 1 else (sb if B > 1 else heads * dim)
    if row < heads * dim or (N > 1 and B > 1 and sb != N * sn):
        raise ValueError(f"{name}: tokens must be evenly spaced and must not overlap")
    return row


def _check_rows(cache: KVCache, name: str, t, B: int, N: int, heads: int) -> int:
    if t.shape != (B, N, heads, cache._dim) or t.device != cache._device:
        raise ValueError(f"{name} must be [{B}, {N}, {heads}, {cache._dim}] on the cache's device")
    return _token_stride(name, t, heads, cache._dim)


def _call(device, fn, *args) -> None:
    """One library call on the device's current stream (the last argument)."""
    st = torch._C._cuda_getCurrentRawStream(device.index)  # torch.cuda.current_stream(device), without its object
    if device.index != torch._C._cuda_getDevice():
        with torch.cuda.device(device):
            rc = fn(*args, st)
    else:
        rc = fn(*args, st)
    if rc != 0:
        raise SpecVerifyError(rc, strerror(rc))


def _workspace(cache: KVCache, need: int, workspace):
    """A workspace of at least `need` bytes: the one given, if it is large enough, or a new one; and its bytes."""
    if need == 0:
        raise SpecVerifyError(-2, strerror(-2))
    have = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if have < need:
        return torch.empty(need, dtype=torch.uint8, device=cache._device), need
    if workspace.device != cache._device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the cache's device")
    return workspace, have


def kv_evict_workspace_size(cache: KVCache, B: int, max_pages: int) -> int:
    """Workspace bytes of kv_evict for page tables of max_pages columns (0: invalid sizes)."""
    return int(load().spec_kv_evict_workspace_size(_descriptor(cache, 16, max_pages), B))


def kv_append(cache: KVCache, page_table, k, v, lengths, *, counts=None, index=None, out_lengths=None):
    """Quantise tokens into the cache behind each sequence's lengths[b] cached
    ones (spec_kv_append).

    k and v [B, N, heads, dim] (bf16 or fp32; a slice of a fused projection's
    rows will do), page_table [B, max_pages], lengths [B] and optionally
    counts [B] (tokens of each sequence) and index [B, N] (which tokens, up to
    the first entry outside [0, N): the path of verify_tree_greedy), int32.
    Returns the tokens cached after the call, [B] int32 (out_lengths if given,
    which overlaps none of the other int32 tensors; lengths itself is left as
    it is, so every layer can pass it).  The cache holds no gradients."""
    _check_table(cache, page_table)
    B, width = page_table.shape
    if k.dim() != 4:
        raise ValueError("k must be [B, N, heads, dim]")
    N, heads = k.shape[1], cache._heads
    row = _check_rows(cache, "k", k, B, N, heads)
    if _check_rows(cache, "v", v, B, N, heads) != row or v.dtype != k.dtype:
        raise ValueError("k and v must have the same dtype and strides")
    _check_ints(cache, (B,), "lengths", lengths)
    if counts is not None:
        _check_ints(cache, (B,), "counts", counts)
    if index is not None:
        _check_ints(cache, (B, N), "index", index)
    if out_lengths is None:
        out_lengths = torch.empty_like(lengths)
    else:
        _check_ints(cache, (B,), "out_lengths", out_lengths)
        at = out_lengths.data_ptr()
        for name, t in (("lengths", lengths), ("counts", counts), ("index", index), ("page_table", page_table)):
            if t is not None and t.data_ptr() < at + 4 * B and at < t.data_ptr() + 4 * t.numel():
                raise ValueError(f"out_lengths must not overlap {name}")
    _call(cache._device, load().spec_kv_append, _descriptor(cache, page_table.data_ptr(), width), k.data_ptr(),
          v.data_ptr(), row, lengths.data_ptr(), _ptr(counts), _ptr(index), B, N, out_lengths.data_ptr(),
          _dtype_code(k.dtype))
    return out_lengths


def kv_read(cache: KVCache, page_table, lengths, T: int, *, starts=None, dtype=None):
    """Cached tokens back as values (spec_kv_read): positions starts[b] ..
    starts[b] + T - 1 (from 0 without starts) of every sequence.  Returns (k,
    v), each [B, T, heads, dim] in dtype (torch.bfloat16, the default, or
    torch.float32), 0 at and behind lengths[b]."""
    _check_table(cache, page_table)
    B, width = page_table.shape
    if T < 1:
        raise ValueError("T must be at least 1")
    _check_ints(cache, (B,), "lengths", lengths)
    if starts is not None:
        _check_ints(cache, (B,), "starts", starts)
    dtype = torch.bfloat16 if dtype is None else dtype
    code = _dtype_code(dtype)
    k = torch.empty((B, T, cache._heads, cache._dim), dtype=dtype, device=cache._device)
    v = torch.empty_like(k)
    _call(cache._device, load().spec_kv_read, _descriptor(cache, page_table.data_ptr(), width), _ptr(starts),
          lengths.data_ptr(), B, T, k.data_ptr(), v.data_ptr(), code)
    return k, v


def kv_attention_workspace_size(cache: KVCache, B: int, N: int, Hq: int, max_pages: int) -> int:
    """Workspace bytes of kv_attention for page tables of max_pages columns (0: invalid sizes)."""
    # the library reads the table's address only to see that there is one
    return int(load().spec_kv_attention_workspace_size(_descriptor(cache, 16, max_pages), B, N, Hq))


def kv_attention(cache: KVCache, page_table, q, lengths, k_new=None, v_new=None, *, parents=None, num_nodes=None,
                 scale: Optional[float] = None, return_lse: bool = False, workspace=None):
    """Attention of N nodes per sequence over the cache and over the nodes
    themselves (spec_kv_attention).

    q [B, N, Hq, dim], k_new and v_new [B, N, heads, dim] (both or neither;
    bf16 or fp32), Hq a multiple of heads; lengths [B] cached tokens,
    parents [B, N] the nodes' tree (None: a chain), num_nodes [B] the nodes of
    each sequence, int32; scale defaults to dim ** -0.5.  Returns out [B, N,
    Hq, dim] and, when asked, lse [B, N, Hq] float32.  Forward only: a
    backward pass through the results raises NotImplementedError."""
    _check_table(cache, page_table)
    B, width = page_table.shape
    if q.dim() != 4:
        raise ValueError("q must be [B, N, Hq, dim]")
    _, N, Hq, dim = q.shape
    q_row = _check_rows(cache, "q", q, B, N, Hq)
    if (k_new is None) != (v_new is None):
        raise ValueError("k_new and v_new go together")
    kv_row = 0
    if k_new is not None:
        heads = cache._heads
        kv_row = _check_rows(cache, "k_new", k_new, B, N, heads)
        if _check_rows(cache, "v_new", v_new, B, N, heads) != kv_row or k_new.dtype != q.dtype or \
                v_new.dtype != q.dtype:
            raise ValueError("k_new and v_new must have the same strides, and q's dtype")
    elif parents is not None:
        raise ValueError("parents needs k_new and v_new")
    _check_ints(cache, (B,), "lengths", lengths)
    if num_nodes is not None:
        _check_ints(cache, (B,), "num_nodes", num_nodes)
    if parents is not None:
        _check_ints(cache, (B, N), "parents", parents)
    code = _dtype_code(q.dtype)
    kv = _descriptor(cache, page_table.data_ptr(), width)
    lib = load()
    workspace, have = _workspace(cache, lib.spec_kv_attention_workspace_size(kv, B, N, Hq), workspace)
    out = torch.empty((B, N, Hq, dim), dtype=q.dtype, device=cache._device)
    lse = torch.empty((B, N, Hq), dtype=torch.float32, device=cache._device) if return_lse else None
    _call(cache._device, lib.spec_kv_attention, kv, q.data_ptr(), q_row, _ptr(k_new), _ptr(v_new), kv_row,
          lengths.data_ptr(), _ptr(num_nodes), _ptr(parents), dim ** -0.5 if scale is None else float(scale), B, N,
          Hq, out.data_ptr(), _ptr(lse), code, workspace.data_ptr(), have)
    results = _forward_only((out, lse) if return_lse else (out,), (q, k_new, v_new))
    return results if return_lse else results[0]


def _check_weights(cache: KVCache, page_table, name: str, t) -> None:
    B, width = page_table.shape
    if t.dtype is not torch.float32 or t.dim() != 3 or t.shape[:2] != (B, cache._heads) or t.device != cache._device or \
            not t.is_contiguous() or t.shape[2] < width * cache._page:
        raise ValueError(f"{name} must be a contiguous float32 [{B}, {cache._heads}, capacity] tensor on the cache's "
                         f"device, capacity at least {width * cache._page}")


def kv_weights(cache: KVCache, page_table, q, lse, lengths, weights, k_new=None, *, counts=None, index=None,
               scale: Optional[float] = None, out=None):
    """Add to weights the attention weight that cached tokens gather from the
    nodes a round keeps (spec_kv_weights).

    q [B, N, Hq, dim] and k_new [B, N, heads, dim] as for kv_attention, lse [B,
    N, Hq] as it returns it (infinite: a query that weighs nothing), lengths [B] the
    tokens cached before the round,
    counts [B] and index [B, N] the kept nodes as for kv_append; weights [B,
    heads, capacity] float32 by cached position, capacity at least max_pages *
    page_size.  Kept nodes get their own weights behind the cached positions
    when k_new is given.  Works in weights itself, or into `out` (positions
    behind are left as they were), which overlaps no other tensor of the call.
    Returns the tensor written, without gradients."""
    _check_table(cache, page_table)
    B, width = page_table.shape
    if q.dim() != 4:
        raise ValueError("q must be [B, N, Hq, dim]")
    _, N, Hq, dim = q.shape
    q_row = _check_rows(cache, "q", q, B, N, Hq)
    k_row = 0
    if k_new is not None:
        k_row = _check_rows(cache, "k_new", k_new, B, N, cache._heads)
        if k_new.dtype != q.dtype:
            raise ValueError("k_new must have q's dtype")
    if lse.dtype is not torch.float32 or lse.shape != (B, N, Hq) or lse.device != cache._device or \
            not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous float32 {[B, N, Hq]} tensor on the cache's device")
    _check_ints(cache, (B,), "lengths", lengths)
    if counts is not None:
        _check_ints(cache, (B,), "counts", counts)
    if index is not None:
        _check_ints(cache, (B, N), "index", index)
    _check_weights(cache, page_table, "weights", weights)
    if out is None:
        out = weights
    else:
        _check_weights(cache, page_table, "out", out)
        if out.shape != weights.shape:
            raise ValueError("out must have weights' shape")
    if out.requires_grad:
        raise ValueError("weights that are written must not require gradients")
    _call(cache._device, load().spec_kv_weights, _descriptor(cache, page_table.data_ptr(), width), q.data_ptr(), q_row,
          lse.data_ptr(), _ptr(k_new), k_row, lengths.data_ptr(), _ptr(counts), _ptr(index),
          dim ** -0.5 if scale is None else float(scale), B, N, Hq, weights.data_ptr(), out.data_ptr(), out.shape[2],
          _dtype_code(q.dtype))
    return out


def kv_evict(cache: KVCache, page_table, lengths, weights, new_pages, budget: int, recent: int, *,
             limit: Optional[int] = None, return_kept: bool = False, workspace=None):
    """Cut sequences of more than limit (default: budget) cached tokens down
    to budget (spec_kv_evict): every head keeps its last `recent` positions and
    the heaviest of the others, in order, in the pages new_pages[b].

    weights [B, heads, capacity] float32 by cached position; new_pages [B,
    ceil(budget / page_size)] int32, pages that no table holds.  Returns
    (page_table, lengths, weights) as they are after the call, in new tensors,
    and when asked the kept positions [B, heads, budget] int32 (-1 where a
    sequence was not cut).  The table rows of the sequences that were cut hold
    their new pages and -1 behind: kv_append takes tokens up to the last of these
    only, until the rows are given more.  The old pages can be used again once the
    call's work is done."""
    _check_table(cache, page_table)
    B, width = page_table.shape
    limit = budget if limit is None else limit
    if budget < 1 or budget > width * cache._page or recent < 0 or recent > budget or limit < budget:
        raise ValueError("0 <= recent <= budget <= limit, 1 <= budget <= max_pages * page_size: got "
                         f"{recent}, {budget}, {limit}")
    _check_ints(cache, (B,), "lengths", lengths)
    _check_weights(cache, page_table, "weights", weights)
    _check_ints(cache, (B, -(-budget // cache._page)), "new_pages", new_pages)
    kv = _descriptor(cache, page_table.data_ptr(), width)
    lib = load()
    workspace, have = _workspace(cache, lib.spec_kv_evict_workspace_size(kv, B), workspace)
    out_table, out_lengths, out_weights = torch.empty_like(page_table), torch.empty_like(lengths), torch.empty_like(weights)
    kept = torch.empty((B, cache._heads, budget), dtype=torch.int32, device=cache._device)
    _call(cache._device, lib.spec_kv_evict, kv, lengths.data_ptr(), weights.data_ptr(), weights.shape[2],
          new_pages.data_ptr(), budget, recent, min(limit, 2 ** 31 - 1), B, out_table.data_ptr(), out_lengths.data_ptr(),
          out_weights.data_ptr(), kept.data_ptr(), workspace.data_ptr(), have)
    return (out_table, out_lengths, out_weights) + ((kept,) if return_kept else ())
