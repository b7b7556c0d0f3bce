"""Paged key-value cache: append, attention of one new token or of a tree of
drafted ones, acceptance of drafts, eviction, page tables.

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
from typing import NamedTuple

from . import _lib

__all__ = ["PagedCache", "Reservation", "cache_accept", "cache_append", "cache_append_packed", "cache_attend",
           "cache_attend_tree", "cache_attend_workspace", "cache_evict", "cache_reserve"]

_STRIDES = struct.Struct("@3q")                      # int64_t[3]
_PAIR = struct.Struct("@2q")
_QUERY = struct.Struct("@PPiiqqqqPPqifPqPqqPq")     # lc_cache_query
_TREE = struct.Struct("@PP4i6q3PqfP2qPq")            # lc_cache_tree
_RESERVATION = struct.Struct("@PP2q10Pq4i")          # lc_cache_reservation
_EVICTION = struct.Struct("@PPqqiiPqqPqqPPq")        # lc_cache_eviction
# of torch, known once a cache exists
_TYPES = None  # dtype -> lc_cache_type
_BYTES = _BOOL = _I32 = _I64 = _F32 = None
_CURRENT = None  # raw handle of a device's current stream (torch.cuda.current_stream() builds an object, 3 us)
_DEVICE = None   # the current device's index (torch.cuda.current_device() takes twice as long)
_GRAD = None     # whether gradients are recorded


def _types():
    global _TYPES, _BYTES, _BOOL, _I32, _I64, _F32, _CURRENT, _DEVICE, _GRAD
    if _TYPES is None:
        import torch
        _BYTES, _BOOL, _I32, _I64, _F32 = torch.uint8, torch.bool, torch.int32, torch.int64, torch.float32
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

    def tree_workspace_bytes(self, n_q_heads: int, drafts: int) -> int:
        key = ("tree", n_q_heads, drafts)
        n = self._workspace_bytes.get(key)
        if n is None:  # (0 for refused arguments: the call says why)
            n = max(0, int(_lib.lib().lc_cache_attend_tree_workspace(self._ref, n_q_heads, drafts)))
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


def cache_append_packed(cache: PagedCache, k, v, slots, stream=None):
    """Writes packed tokens into the slots that ``cache_reserve`` gave them.

    ``k``, ``v``: [tokens, kv_heads, head_dim], of the types that ``cache_append``
    takes.  ``slots``: int64 [tokens], page * page_size + row, no two alike; a
    token of -1 is dropped, and so is one outside the pool, which sets the device error word.
    """
    shape = k.shape
    kind = _TYPES.get(k.dtype)
    if len(shape) != 3 or kind is None or kind > 1:
        raise ValueError("new keys and values are [tokens, kv_heads, head_dim] of bfloat16 or float16")
    _tensor(k, "k", k.dtype, (shape[0], cache.n_kv_heads, cache.head_dim), cache.device)
    _tensor(v, "v", k.dtype, shape, cache.device)
    if k.requires_grad or v.requires_grad:
        _no_gradient()
    _tensor(slots, "slots", _I64, (shape[0],), cache.device)
    if stream is not None:
        with _on(stream) as handle:
            return _append_packed(cache, k, v, kind, slots, handle)
    return _append_packed(cache, k, v, kind, slots, _CURRENT(cache._index))


def _append_packed(cache, k, v, kind, slots, handle):
    if _DEVICE() != cache._index:
        _elsewhere(cache)
    status = _lib.lib().lc_cache_append_packed(
        cache._ref, k.data_ptr(), v.data_ptr(), kind, _PAIR.pack(*k.stride()[:2]), _PAIR.pack(*v.stride()[:2]),
        k.shape[0], slots.data_ptr(), handle)
    if status:
        _check(status, "cache_append_packed")


def cache_attend_tree(cache: PagedCache, q, lengths, parents, counts=None, out=None, scale=None, window: int = 0,
                      lse=None, workspace=None, stream=None):
    """Attention of a tree of drafted tokens a sequence over its cached slots; returns ``out``.

    The drafts' keys and values are in the cache already (``cache_append``):
    draft t sits in slot lengths[b] - counts[b] + t.  It sees the slots before the drafts, its
    ancestors' and its own.  ``q``: [seqs, drafts, q_heads, head_dim] of the cache's
    type (bfloat16 for a float8_e4m3fn cache), at most 64 drafts; query head i reads key head
    i // (q_heads // kv_heads).  ``parents``: int32 [seqs, drafts], an earlier draft
    or -1 for those that follow the token before the drafts (a chain: t - 1).
    ``counts``: int32 [seqs], how many drafts a sequence has (default: all); rows past them are left as they
    were (in an ``out`` that is made here: undefined).  ``out``: like ``q``, apart from it.  ``scale``: of the dot
    products, 1 / sqrt(head_dim) by default.  ``window``: how many tokens a draft sees,
    itself, its nearest ancestors and then the newest before the drafts (0: all).
    ``lse``: float32 [seqs, drafts, q_heads] to receive log sum exp, apart from the others.
    ``workspace``: at least ``cache.tree_workspace_bytes(q_heads, drafts)`` bytes; calls that may overlap need one each.
    """
    shape = q.shape
    if len(shape) != 4:
        raise ValueError("q is [seqs, drafts, q_heads, head_dim]")
    device, (n_seqs, drafts, n_q, _) = cache.device, shape
    _tensor(q, "q", cache.io_dtype, (cache.n_seqs, drafts, n_q, cache.head_dim), device)
    if q.requires_grad:
        _no_gradient()
    _tensor(lengths, "lengths", _I32, cache._seqs, device)
    _tensor(parents, "parents", _I32, (n_seqs, drafts), device)
    if counts is not None:
        _tensor(counts, "counts", _I32, cache._seqs, device)
    if lse is not None:
        _tensor(lse, "lse", _F32, (n_seqs, drafts, n_q), device)
    if out is not None:
        _tensor(out, "out", q.dtype, shape, device)
    if workspace is not None and (workspace.device != device or not workspace.is_contiguous()):
        raise ValueError("the workspace must be contiguous and on the cache's device")
    if stream is not None:
        with _on(stream) as handle:
            return _attend_tree(cache, q, lengths, parents, counts, out, scale, window, lse, workspace, handle)
    return _attend_tree(cache, q, lengths, parents, counts, out, scale, window, lse, workspace, _CURRENT(cache._index))


def _attend_tree(cache, q, lengths, parents, counts, out, scale, window, lse, workspace, handle):
    if _DEVICE() != cache._index:
        _elsewhere(cache)
    n, t, h, d = q.shape
    if out is None:
        out = cache._empty((n, t, h, d), (t * h * d, h * d, d, 1), q.dtype)
    if workspace is None:
        workspace = cache._empty((cache.tree_workspace_bytes(h, t),), (1,), _BYTES)
    l0 = l1 = logs = 0
    if lse is not None:
        logs, (l0, l1, _) = lse.data_ptr(), lse.stride()
    a = _TREE.pack(q.data_ptr(), out.data_ptr(), _TYPES[q.dtype], h, t, window if window < 0x7fffffff else 0x7fffffff,
                   *q.stride()[:3], *out.stride()[:3], lengths.data_ptr(), 0 if counts is None else counts.data_ptr(),
                   parents.data_ptr(), parents.stride(0), cache.scale if scale is None else scale, logs, l0, l1,
                   workspace.data_ptr(), workspace.numel() * workspace.element_size())
    status = _lib.lib().lc_cache_attend_tree(cache._ref, a, handle)
    if status:
        _check(status, "cache_attend_tree")
    return out


def cache_accept(cache: PagedCache, lengths, counts, path, new_lengths=None, stream=None):
    """Keeps the accepted drafts of each sequence; returns the new lengths.

    ``path``: int32 [seqs, most], at most 64 columns: a sequence's accepted drafts in rising order, ended by -1.
    The i-th of them moves from slot lengths[b] - counts[b] + path[b, i] to slot
    lengths[b] - counts[b] + i.  ``counts``: int32 [seqs], how many drafts a sequence
    has (None: as many as ``path`` has columns).  ``new_lengths``: an int32 [seqs] tensor to receive lengths -
    counts + the accepted ones, apart from the inputs and the page table.  A path that does not rise, or
    leaves the drafts, ends there and sets the device error word.  The pages that hold
    the drafts must not be shared with another sequence.
    """
    device, seqs = cache.device, cache._seqs
    _tensor(lengths, "lengths", _I32, seqs, device)
    if counts is not None:
        _tensor(counts, "counts", _I32, seqs, device)
    if path.dim() != 2:
        raise ValueError("path is [seqs, most]")
    _tensor(path, "path", _I32, (cache.n_seqs, path.shape[1]), device)
    if new_lengths is not None:
        _tensor(new_lengths, "new_lengths", _I32, seqs, device)
    if stream is not None:
        with _on(stream) as handle:
            return _accept(cache, lengths, counts, path, new_lengths, handle)
    return _accept(cache, lengths, counts, path, new_lengths, _CURRENT(cache._index))


def _accept(cache, lengths, counts, path, new_lengths, handle):
    if _DEVICE() != cache._index:
        _elsewhere(cache)
    if new_lengths is None:
        new_lengths = cache._empty(cache._seqs, (1,), _I32)
    status = _lib.lib().lc_cache_accept(cache._ref, lengths.data_ptr(), None if counts is None else counts.data_ptr(),
                                        path.data_ptr(), path.stride(0), path.shape[1], new_lengths.data_ptr(), handle)
    if status:
        _check(status, "cache_accept")
    return new_lengths


class Reservation(NamedTuple):
    """What ``cache_reserve`` returns."""
    table: object      # int32 [seqs, pages_per_seq]
    lengths: object    # int32 [seqs]: lengths with the new tokens of the sequences that are served
    starts: object     # int32 [seqs + 1]: where each sequence's tokens begin among the packed ones
    slots: object      # int64 [max_tokens]: page * page_size + row of every packed token, -1 past the last
    positions: object  # int32 [max_tokens]: its place in its sequence
    seqs: object       # int32 [max_tokens]: its sequence
    n_free: object     # int32 [1]: pages left on the stack


def cache_reserve(page_table, lengths, counts, free, n_free, page_size: int, max_tokens: int, new_table=None,
                  stream=None):
    """Makes a page table hold the pages of lengths + counts tokens a sequence; returns a ``Reservation``.

    ``page_table``: int32 [seqs, pages_per_seq], each row a sequence's pages and then
    -1; changed in place, or written to ``new_table`` where that is given.
    ``lengths``, ``counts``: int32 [seqs], tokens that a sequence has, and new
    ones.  ``free``, ``n_free``: int32 [any] and [1], a stack of free pages and how many it has;
    the stack is changed in place, its new height returned.  Pages past those that a sequence wants (one that
    has ended has length and count 0) go on the stack, then what is missing comes off
    its top, in the sequences' order.  ``max_tokens``: the size of the packed lists.  A
    sequence whose pages do not last, whose tokens pass the table's columns or the
    lists gets none, keeps its pages, and the device error word is set; those behind it
    that need no pages are served all the same.  At most 4096 sequences.
    """
    _types()
    device, shape = page_table.device, page_table.shape
    if page_table.dim() != 2 or not page_table.is_cuda:
        raise ValueError("the page table is int32 [seqs, pages_per_seq] on a CUDA device (there is no CPU path)")
    _tensor(page_table, "page_table", _I32, shape, device)
    _tensor(lengths, "lengths", _I32, shape[:1], device)
    _tensor(counts, "counts", _I32, shape[:1], device)
    if free.dim() != 1:
        raise ValueError("free is int32 [any]")
    _tensor(free, "free", _I32, free.shape, device)
    _tensor(n_free, "n_free", _I32, (1,), device)
    if new_table is not None:
        _tensor(new_table, "new_table", _I32, shape, device)
    page_size, max_tokens = int(page_size), int(max_tokens)
    if _DEVICE() != device.index:
        raise ValueError("the page table is on %s, the current device is cuda:%d" % (device, _DEVICE()))
    if stream is not None:
        with _on(stream) as handle:
            return _reserve(page_table, lengths, counts, free, n_free, page_size, max_tokens, new_table, handle)
    return _reserve(page_table, lengths, counts, free, n_free, page_size, max_tokens, new_table, _CURRENT(device.index))


def _reserve(page_table, lengths, counts, free, n_free, page_size, max_tokens, new_table, handle):
    n, per = page_table.shape
    tokens = max(max_tokens, 0)
    empty = _empty()
    if new_table is None:
        new_table = page_table
    new_lengths, starts = empty((n,), (1,), _I32), empty((n + 1,), (1,), _I32)
    slots, positions, seqs = empty((tokens,), (1,), _I64), empty((tokens,), (1,), _I32), empty((tokens,), (1,), _I32)
    new_n_free = empty((1,), (1,), _I32)
    a = _RESERVATION.pack(page_table.data_ptr(), new_table.data_ptr(), page_table.stride(0), new_table.stride(0),
                          lengths.data_ptr(), counts.data_ptr(), free.data_ptr(), n_free.data_ptr(),
                          new_n_free.data_ptr(), new_lengths.data_ptr(), starts.data_ptr(), slots.data_ptr(),
                          positions.data_ptr(), seqs.data_ptr(), free.shape[0], n, per, page_size, max_tokens)
    status = _lib.lib().lc_cache_reserve(a, handle)
    if status:
        _check(status, "cache_reserve")
    return Reservation(new_table, new_lengths, starts, slots, positions, seqs, new_n_free)


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
