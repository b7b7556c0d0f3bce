"""Attention over whole prompts: packed sequences of different lengths.

Everything runs in the C-ABI library (``include/layout_copy_prompt.h``); this
module marshals arguments and allocates outputs through torch.  There is no
backward pass: inputs that want a gradient are refused.
"""
from __future__ import annotations

import math
import struct

from . import _lib, cache as _cache

__all__ = ["prompt_attend"]

_PROMPT = struct.Struct("@7P2q7if2q2q2q2qq")  # lc_prompt


def _rows(t, name: str, like, heads):
    """Packed rows [tokens, heads, head_dim] of q's type, on q's device, a row's elements adjacent."""
    if t.dim() != 3 or t.dtype is not like.dtype or t.shape[2] != like.shape[2] or (heads and t.shape[1] != heads):
        raise ValueError("%s must be [tokens, heads, head_dim] of q's type and head_dim%s, got %s of shape %r"
                         % (name, " with %d heads" % heads if heads else "", t.dtype, tuple(t.shape)))
    if t.device != like.device:
        raise ValueError("%s is on %s, q on %s" % (name, t.device, like.device))
    if t.shape[2] > 1 and t.stride(2) != 1:
        raise ValueError("%s: the elements of the last mode must be adjacent" % name)


def _list(t, name: str, dtype, shape, device):
    if t.dtype is not dtype or t.shape != shape or t.device != device or (shape[-1] > 1 and t.stride(-1) != 1):
        raise ValueError("%s must be %s of shape %r on %s with adjacent elements, got %s of shape %r on %s"
                         % (name, dtype, tuple(shape), device, t.dtype, tuple(t.shape), t.device))


def prompt_attend(q, k, v, starts, k_starts=None, causal: bool = True, window: int = 0, scale=None, out=None, lse=None,
                  stream=None):
    """Attention of packed sequences over their own keys and values; returns ``out``.

    ``q``: [tokens, q_heads, head_dim] of bfloat16 or float16, ``k`` and ``v``:
    [keys, kv_heads, head_dim] of its type; query head i reads key head i //
    (q_heads // kv_heads).  ``starts``: int32 [seqs + 1], sequence b is the
    tokens starts[b] .. starts[b + 1] - 1.  ``k_starts``: the same of the keys
    (default: ``starts``); a sequence with more keys than queries is a later
    piece of a prompt, its queries the last of its tokens.  ``causal``: keys
    after a query are not seen.  ``window``: of the keys up to a query's own
    place only the newest so many are seen (0: all).  ``scale``: of the dot products, 1 /
    sqrt(head_dim) by default.  ``out``: like ``q``, and either ``q`` itself or
    apart from it, ``k`` and ``v``.  ``lse``: float32 [tokens, q_heads] to receive log sum exp.
    A query with nothing to see gives zeros (lse: -inf); rows that are no sequence's
    are left as they were (in an ``out`` that is made here: undefined).  head_dim is a
    multiple of 8 up to 256 and rows lie on 16-byte boundaries.  The call runs on the current device, which has to be the
    tensors'.  What is rounded on the way is in ``include/layout_copy_prompt.h``.
    """
    kinds = _cache._types()
    if q.dim() != 3 or kinds.get(q.dtype, 2) > 1:
        raise ValueError("q is [tokens, q_heads, head_dim] of bfloat16 or float16")
    if not q.is_cuda:
        raise ValueError("prompt_attend needs CUDA tensors (there is no CPU path)")
    device = q.device
    tokens, heads, dim = q.shape
    _rows(q, "q", q, heads)
    _rows(k, "k", q, 0)
    _rows(v, "v", q, k.shape[1])
    if v.shape[0] != k.shape[0]:
        raise ValueError("k and v must have as many rows, got %d and %d" % (k.shape[0], v.shape[0]))
    if q.requires_grad or k.requires_grad or v.requires_grad:
        _cache._no_gradient()
    if starts.dim() != 1 or starts.shape[0] < 1:
        raise ValueError("starts is int32 [seqs + 1]")
    _list(starts, "starts", _cache._I32, starts.shape, device)
    if k_starts is not None:
        _list(k_starts, "k_starts", _cache._I32, starts.shape, device)
    elif k.shape[0] != tokens:
        raise ValueError("k has %d rows and q %d: sequences with other keys than queries need k_starts"
                         % (k.shape[0], tokens))
    if out is not None:
        _rows(out, "out", q, heads)
        if out.shape[0] != tokens:
            raise ValueError("out must have q's shape %r, got %r" % (tuple(q.shape), tuple(out.shape)))
    if lse is not None:
        _list(lse, "lse", _cache._F32, (tokens, heads), device)
    index = device.index
    if _cache._DEVICE() != index:
        raise ValueError("q is on %s, the current device is cuda:%d: outputs are made and kernels run there "
                         "(torch.cuda.set_device, or a stream of the tensors' device)" % (device, _cache._DEVICE()))
    if stream is not None:
        with _cache._on(stream) as handle:
            return _attend(q, k, v, starts, k_starts, causal, window, scale, out, lse, handle)
    return _attend(q, k, v, starts, k_starts, causal, window, scale, out, lse, _cache._CURRENT(index))


def _attend(q, k, v, starts, k_starts, causal, window, scale, out, lse, handle):
    tokens, heads, dim = q.shape
    if out is None:
        out = _cache._empty()((tokens, heads, dim), (heads * dim, dim, 1), q.dtype)
    logs, lse_stride = (0, 0) if lse is None else (lse.data_ptr(), lse.stride(0))
    a = _PROMPT.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), logs, starts.data_ptr(),
                     0 if k_starts is None else k_starts.data_ptr(), tokens, k.shape[0], _cache._TYPES[q.dtype],
                     starts.shape[0] - 1, heads, k.shape[1], dim, 1 if causal else 0,
                     window if window < 0x7fffffff else 0x7fffffff, 1.0 / math.sqrt(dim) if scale is None else scale,
                     *q.stride()[:2], *k.stride()[:2], *v.stride()[:2], *out.stride()[:2], lse_stride)
    status = _lib.lib().lc_prompt_attend(a, handle)
    if status:
        _cache._check(status, "prompt_attend")
    return out
