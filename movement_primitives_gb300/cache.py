"""Paged key-value cache: append, attention of one new token, eviction.

A cache is a pool of pages seen as [page, kv_head, slot, dim] through its
strides (a [page, slot, kv_head, dim] pool is passed as its ``transpose(1,
2)``) and a page table naming each sequence's pages.  Everything runs in the
C-ABI library (``include/layout_copy_cache.h``); this module marshals
arguments and allocates outputs and workspaces through torch.  There is no
backward pass: inputs that want a gradient are refused.
"""
from __future__ import annotations

import ctypes
import math
import struct

from . import _lib

__all__ = ["PagedCache", "cache_append", "cache_attend", "cache_attend_workspace", "cache_evict"]

_STRIDES = struct.Struct("@3q")                      # int64_t[3]
_QUERY = struct.Struct("@PPiiqqqqPPqifPqPqqPq")     # lc_cache_query
_EVICTION = struct.Struct("@PPqqiiPqqPqqPPq")        # lc_cache_eviction
# of torch, known once a cache exists
_TYPES = None  # dtype -> lc_cache_type
_BYTES = _BOOL = _I32 = _F32 = None
_CURRENT = None  # raw handle of a device's current stream (torch.cuda.current_stream() builds an object, 3 us)
_DEVICE = None   # the current device's index (torch.cuda.current_device() takes twice as long)
_GRAD = None     # whether gradients are recorded


def _types():
    global _TYPES, _BYTES, _BOOL, _I32, _F32, _CURRENT, _DEVICE, _GRAD
    if _TYPES is None:
        import torch
        _BYTES, _BOOL, _I32, _F32 = torch.uint8, torch.bool, torch.int32, torch.float32
        _CURRENT = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda index: torch.cuda.current_stream(index).cuda_stream)
        _DEVICE = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        _GRAD = torch.is_grad_enabled
        _TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float8_e4m3fn: 2}
    return _TYPES


def _check(status: int, what: str) -> None:
    if status != 0:
        from . import LayoutCopyError
        raise LayoutCopyError(status, what)


def _allocator():
    """``empty(shape, strides, dtype)`` on the current device and stream.  torch's direct binding where it has it:
    torch.empty takes 3.5 us more a call, as long as one of the library's launches.  It comes from the same caching
    allocator (streams, graphs and memory pools included) and passes by the dispatcher, whose modes see nothing of it
    and fill nothing: every element of an output is written by the kernels."""
    import torch
    direct = getattr(getattr(torch._C._dynamo, "guards", None), "_empty_strided_cuda", None) \
        if hasattr(torch._C, "_dynamo") else None
    if direct is not None:
        return direct
    return lambda shape, strides, dtype: torch.empty_strided(shape, strides, dtype=dtype, device="cuda")


_EMPTY = None


def _empty():
    """The allocator, looked up once."""
    global _EMPTY
    if _EMPTY is None:
        _EMPTY = _allocator()
    return _EMPTY


def _elsewhere(cache):
    raise ValueError("the cache is on %s, the current device is cuda:%d: outputs are made and kernels run there "
                     "(torch.cuda.set_device, or a stream of the cache's device)" % (cache.device, _DEVICE()))


class _on:
    """Runs allocations on the stream the kernels will use, so that torch's
    allocator hands the memory out in that stream's order."""

    def __init__(self, stream):
        import torch
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
        self.ctx, self.handle = torch.cuda.stream(stream), stream.cuda_stream

    def __enter__(self):
        self.ctx.__enter__()
        return self.handle

    def __exit__(self, *exc):
        self.ctx.__exit__(*exc)


def _no_gradient():
    if _GRAD():
        raise ValueError("no operator of the cache has a gradient: detach its inputs or call it under torch.no_grad()")


def _tensor(t, name: str, dtype, shape, device):
    """A tensor of that type and shape on the cache's device whose last mode's elements are adjacent."""
    if t.dtype is dtype and t.shape == shape and t.device == device and (
            t.is_contiguous() or shape[-1] <= 1 or t.stride(-1) == 1):
        return t
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %r, got %r" % (name, tuple(shape), tuple(t.shape)))
    if t.device != device:
        raise ValueError("%s is on %s, the cache on %s" % (name, t.device, device))
    raise ValueError("%s: the elements of the last mode must be adjacent" % name)


class PagedCache:
    """Pools of pages and a page table.

    ``k``, ``v``: CUDA tensors [pages, kv_heads, page_size, head_dim] of
    bfloat16, float16 or float8_e4m3fn, any strides with adjacent elements in
    the last mode.  ``page_table``: int32 [seqs, pages_per_seq]; entries past a
    sequence's pages are never read.  ``k_scale``, ``v_scale``: float32 [pages,
    kv_heads, page_size] for float8_e4m3fn pools (value = code * scale).  The
    tensors are kept by reference: what they hold may change between calls,
    their memory may not.  The operators run on the current device, which has
    to be theirs.  Kernels and workspaces are chosen by ``capacity``, the slots
    that the table has columns for: where sequences are known to be far shorter, a
    cache over ``page_table[:, :columns]`` (masks and scores of as many slots) is
    faster and takes less memory.
    """

    def __init__(self, k, v, page_table, k_scale=None, v_scale=None):
        import torch
        if not k.is_cuda:
            raise ValueError("a cache needs CUDA tensors (there is no CPU path)")
        if k.dim() != 4 or page_table.dim() != 2:
            raise ValueError("pools are [pages, kv_heads, page_size, head_dim], the table [seqs, pages_per_seq]")
        if k.dtype not in _types():
            raise ValueError("pools are bfloat16, float16 or float8_e4m3fn, got %s" % k.dtype)
        _tensor(k, "k", k.dtype, tuple(k.shape), k.device)
        _tensor(v, "v", k.dtype, tuple(k.shape), k.device)
        _tensor(page_table, "page_table", torch.int32, tuple(page_table.shape), k.device)
        q8 = k.dtype == torch.float8_e4m3fn
        if q8 != (k_scale is not None) or q8 != (v_scale is not None):
            raise ValueError("k_scale and v_scale belong to float8_e4m3fn pools, and only to them")
        c = _lib.CPagedCache()
        if q8:
            for name, s in (("k_scale", k_scale), ("v_scale", v_scale)):
                if s.dtype != torch.float32 or tuple(s.shape) != tuple(k.shape[:3]) or s.device != k.device:
                    raise ValueError("%s must be float32 of shape %r on the pools' device" % (name, tuple(k.shape[:3])))
            c.k_scale, c.v_scale = k_scale.data_ptr(), v_scale.data_ptr()
            c.k_scale_stride[:] = k_scale.stride()
            c.v_scale_stride[:] = v_scale.stride()
        c.k, c.v, c.page_table = k.data_ptr(), v.data_ptr(), page_table.data_ptr()
        c.table_stride = page_table.stride(0)
        c.n_pages, c.n_kv_heads, c.page_size, c.head_dim = k.shape
        c.n_seqs, c.pages_per_seq = page_table.shape
        c.type = _types()[k.dtype]
        c.k_stride[:] = k.stride()[:3]
        c.v_stride[:] = v.stride()[:3]
        self._c, self._ref = c, ctypes.byref(c)
        self._workspace_bytes = {}
        self.k, self.v, self.page_table, self.k_scale, self.v_scale = k, v, page_table, k_scale, v_scale
        self.device, self.dtype = k.device, k.dtype
        self.n_seqs, self.pages_per_seq = page_table.shape
        self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = k.shape
        self.capacity = self.page_size * self.pages_per_seq
        self._empty = _empty()
        self._index, self._seqs = k.device.index, (self.n_seqs,)
        self.scale = 1.0 / math.sqrt(self.head_dim)
        self.io_dtype = torch.bfloat16 if q8 else k.dtype

    def workspace_bytes(self, n_q_heads: int, with_scores: bool) -> int:
        key = (n_q_heads, with_scores)
        n = self._workspace_bytes.get(key)
        if n is None:
            n = int(_lib.lib().lc_cache_attend_workspace(self._ref, n_q_heads, int(with_scores)))
            if n < 0:
                raise ValueError("a cache of %d key heads cannot take %d query heads (or is itself refused)"
                                 % (self.n_kv_heads, n_q_heads))
            self._workspace_bytes[key] = n
        return n

    def evict_workspace_bytes(self, budget: int) -> int:
        n = self._workspace_bytes.get(budget)
        if n is None:  # (0 for a refused budget: the call says why)
            n = max(0, int(_lib.lib().lc_cache_evict_workspace(self._ref, budget)))
            self._workspace_bytes[budget] = n
        return n


def cache_append(cache: PagedCache, k, v, lengths, counts=None, new_lengths=None, stream=None):
    """Writes new tokens after each sequence's ``lengths``; returns the new lengths.

    ``k``, ``v``: [seqs, tokens, kv_heads, head_dim] of the cache's type, or of
    bfloat16 / float16 for a float8_e4m3fn cache (each row is quantised with a
    scale of its own).  ``lengths``: int32 [seqs].  ``counts``: int32 [seqs],
    how many of the tokens are a sequence's (default: all).  ``new_lengths``:
    an int32 [seqs] tensor to receive lengths + counts, apart from ``lengths``
    and ``counts``.  Tokens past a sequence's capacity are dropped and set the device
    error word (``last_device_error``).
    """
    shape = k.shape
    kind = _TYPES.get(k.dtype)
    if len(shape) != 4 or kind is None or kind > 1:
        raise ValueError("new keys and values are [seqs, tokens, kv_heads, head_dim] of bfloat16 or float16")
    device, seqs = cache.device, cache._seqs
    _tensor(k, "k", k.dtype, (cache.n_seqs, shape[1], cache.n_kv_heads, cache.head_dim), device)
    _tensor(v, "v", k.dtype, shape, device)
    if k.requires_grad or v.requires_grad:
        _no_gradient()
    _tensor(lengths, "lengths", _I32, seqs, device)
    if counts is not None:
        _tensor(counts, "counts", _I32, seqs, device)
    if new_lengths is not None:
        _tensor(new_lengths, "new_lengths", _I32, seqs, device)
    if stream is not None:
        with _on(stream) as handle:
            return _append(cache, k, v, kind, shape[1], counts, lengths, new_lengths, handle)
    return _append(cache, k, v, kind, shape[1], counts, lengths, new_lengths, _CURRENT(cache._index))


def _append(cache, k, v, kind, n_new, counts, lengths, new_lengths, handle):
    if _DEVICE() != cache._index:
        _elsewhere(cache)
    if new_lengths is None:
        new_lengths = cache._empty(cache._seqs, (1,), _I32)
    status = _lib.lib().lc_cache_append(
        cache._ref, k.data_ptr(), v.data_ptr(), kind, _STRIDES.pack(*k.stride()[:3]), _STRIDES.pack(*v.stride()[:3]),
        n_new, None if counts is None else counts.data_ptr(), lengths.data_ptr(), new_lengths.data_ptr(), handle)
    if status:
        _check(status, "cache_append")
    return new_lengths


def cache_attend_workspace(cache: PagedCache, n_q_heads: int, with_scores: bool = False, stream=None):
    """A workspace for ``cache_attend`` calls that do not overlap."""
    import torch
    n = cache.workspace_bytes(n_q_heads, with_scores)
    if stream is not None:
        with _on(stream):
            return torch.empty(n, dtype=torch.uint8, device=cache.device)
    return torch.empty(n, dtype=torch.uint8, device=cache.device)


def cache_attend(cache: PagedCache, q, lengths, out=None, scale=None, window: int = 0, mask=None, lse=None,
                 scores=None, workspace=None, stream=None):
    """Attention of one new token a sequence over its cached slots; returns ``out``.

    ``q``: [seqs, q_heads, head_dim] of the cache's type (bfloat16 for a
    float8_e4m3fn cache); query head i reads key head i // (q_heads //
    kv_heads).  ``out``: like ``q``, and either ``q`` itself or apart from it.
    ``scale``: of the dot products, 1 / sqrt(head_dim) by default.
    ``window``: only the newest so many slots are seen (0: all).  ``mask``:
    bool or uint8 [seqs, capacity], slots of a zero are not seen.  ``lse``:
    float32 [seqs, q_heads] to receive log sum exp.  ``scores``: float32
    [seqs, kv_heads, capacity]; each slot's weight, summed over its query heads, is
    added to it.  A row with no slot seen gives zeros (lse: -inf).  Sums are
    float32 and the output is rounded once; what is rounded on the way is in
    ``include/layout_copy_cache.h``.
    """
    shape = q.shape
    if len(shape) != 3:
        raise ValueError("q is [seqs, q_heads, head_dim]")
    n_q, n_seqs, device = shape[1], cache.n_seqs, cache.device
    _tensor(q, "q", cache.io_dtype, (n_seqs, n_q, cache.head_dim), device)
    if q.requires_grad:
        _no_gradient()
    _tensor(lengths, "lengths", _I32, cache._seqs, device)
    if mask is not None:
        if mask.dtype is not _BOOL and mask.dtype is not _BYTES:
            raise ValueError("mask must be bool or uint8, got %s" % mask.dtype)
        _tensor(mask, "mask", mask.dtype, (n_seqs, cache.capacity), device)
    if lse is not None:
        _tensor(lse, "lse", _F32, (n_seqs, n_q), device)
    if scores is not None:
        _tensor(scores, "scores", _F32, (n_seqs, cache.n_kv_heads, cache.capacity), device)
    if out is not None:
        _tensor(out, "out", q.dtype, shape, device)
    if workspace is not None and (workspace.device != device or not workspace.is_contiguous()):
        raise ValueError("the workspace must be contiguous and on the cache's device")
    if stream is not None:
        with _on(stream) as handle:
            return _attend(cache, q, n_q, lengths, out, scale, window, mask, lse, scores, workspace, handle)
    return _attend(cache, q, n_q, lengths, out, scale, window, mask, lse, scores, workspace, _CURRENT(cache._index))


def _attend(cache, q, n_q, lengths, out, scale, window, mask, lse, scores, workspace, handle):
    if _DEVICE() != cache._index:
        _elsewhere(cache)
    kind = _TYPES[q.dtype]
    if out is None:
        d = cache.head_dim
        out = cache._empty((cache.n_seqs, n_q, d), (n_q * d, d, 1), q.dtype)
    ws, ws_bytes = 0, 0
    if workspace is not None:
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    else:
        ws_bytes = cache.workspace_bytes(n_q, scores is not None)
        if ws_bytes:
            workspace = cache._empty((ws_bytes,), (1,), _BYTES)
            ws = workspace.data_ptr()
    q0, q1, _ = q.stride()
    o0, o1, _ = out.stride()
    # lc_cache_query, packed in one call (a ctypes structure's fields one by one cost several times that)
    masked, mask_stride, logs, lse_stride, sums, s0, s1 = 0, 0, 0, 0, 0, 0, 0
    if mask is not None:
        masked, mask_stride = mask.data_ptr(), mask.stride(0)
    if lse is not None:
        logs, lse_stride = lse.data_ptr(), lse.stride(0)
    if scores is not None:
        sums, (s0, s1, _) = scores.data_ptr(), scores.stride()
    a = _QUERY.pack(q.data_ptr(), out.data_ptr(), kind, n_q, q0, q1, o0, o1, lengths.data_ptr(), masked, mask_stride,
                    window if window < 0x7fffffff else 0x7fffffff, cache.scale if scale is None else scale, logs,
                    lse_stride, sums, s0, s1, ws, ws_bytes)
    status = _lib.lib().lc_cache_attend(cache._ref, a, handle)
    if status:
        _check(status, "cache_attend")
    return out


def cache_evict(cache: PagedCache, lengths, scores, budget: int, recent: int = 0, new_scores=None, kept=None,
                new_lengths=None, stream=None):
    """Cuts sequences of more than ``budget`` slots down to it; returns (kept, new_scores, new_lengths).

    Per key head the ``recent`` newest slots stay, and of the others those of
    the largest ``scores`` (float32 [seqs, kv_heads, capacity]; equal ones:
    the lowest slots).  Their rows move to the front of the sequence's pages
    in their order.  ``kept``: int32 [seqs, kv_heads, budget], the old slot of
    each kept one, then -1.  ``new_scores``: the kept slots' scores, then
    zeros, apart from ``scores``; ``new_lengths``: min(lengths, budget), apart
    from ``lengths``.  The pages a sequence's table
    names must be its own.
    """
    n_seqs, heads, device = cache.n_seqs, cache.n_kv_heads, cache.device
    _tensor(lengths, "lengths", _I32, cache._seqs, device)
    _tensor(scores, "scores", _F32, (n_seqs, heads, cache.capacity), device)
    budget, recent = int(budget), int(recent)
    if kept is not None:
        _tensor(kept, "kept", _I32, (n_seqs, heads, budget), device)
    if new_scores is not None:
        _tensor(new_scores, "new_scores", _F32, scores.shape, device)
    if new_lengths is not None:
        _tensor(new_lengths, "new_lengths", _I32, cache._seqs, device)
    if stream is not None:
        with _on(stream) as handle:
            return _evict(cache, lengths, scores, budget, recent, new_scores, kept, new_lengths, handle)
    return _evict(cache, lengths, scores, budget, recent, new_scores, kept, new_lengths, _CURRENT(cache._index))


def _evict(cache, lengths, scores, budget, recent, new_scores, kept, new_lengths, handle):
    if _DEVICE() != cache._index:
        _elsewhere(cache)
    b, h, cap = cache.n_seqs, cache.n_kv_heads, cache.capacity
    if kept is None:
        n = max(budget, 0)
        kept = cache._empty((b, h, n), (h * n, n, 1), _I32)
    if new_scores is None:
        new_scores = cache._empty((b, h, cap), (h * cap, cap, 1), _F32)
    if new_lengths is None:
        new_lengths = cache._empty((b,), (1,), _I32)
    ws_bytes = cache.evict_workspace_bytes(budget)
    workspace = cache._empty((ws_bytes,), (1,), _BYTES) if ws_bytes else None
    s0, s1, _ = scores.stride()
    k0, k1, _ = kept.stride()
    n0, n1, _ = new_scores.stride()
    a = _EVICTION.pack(lengths.data_ptr(), scores.data_ptr(), s0, s1, budget, recent, kept.data_ptr(), k0, k1,
                       new_scores.data_ptr(), n0, n1, new_lengths.data_ptr(),
                       workspace.data_ptr() if ws_bytes else 0, ws_bytes)
    status = _lib.lib().lc_cache_evict(cache._ref, a, handle)
    if status:
        _check(status, "cache_evict")
    return kept, new_scores, new_lengths
