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


def _rows(t, name: str, dtype, dim: int, device, heads: int):
    """Shape and strides of packed rows [tokens, heads, head_dim] (heads 0: any number) on q's device, a row's elements
    adjacent."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or t.dtype is not dtype or shape[2] != dim or (heads and shape[1] != heads):
        raise ValueError("%s must be [tokens, heads, head_dim] of q's type and head_dim%s, got %s of shape %r"
                         % (name, " with %d heads" % heads if heads else "", t.dtype, tuple(shape)))
    if t.device != device:
        raise ValueError("%s is on %s, q on %s" % (name, t.device, device))
    if dim > 1 and stride[2] != 1:
        raise ValueError("%s: the elements of the last mode must be adjacent" % name)
    return shape, stride


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
    apart from it, ``k`` and ``v``.  ``lse``: float32 [tokens, q_heads] to receive log sum exp, apart from the others.
    A query with nothing to see gives zeros (lse: -inf); rows that are no sequence's
    are left as they were (in an ``out`` that is made here: undefined).  head_dim is a
    multiple of 8 up to 256 and rows lie on 16-byte boundaries.  The call runs on the current device, which has to be the
    tensors'.  What is rounded on the way is in ``include/layout_copy_prompt.h``.
    """
    kind = _cache._types().get(q.dtype, 2)
    if q.dim() != 3 or kind > 1:
        raise ValueError("q is [tokens, q_heads, head_dim] of bfloat16 or float16")
    if not q.is_cuda:
        raise ValueError("prompt_attend needs CUDA tensors (there is no CPU path)")
    device, dtype, shape = q.device, q.dtype, q.shape
    tokens, heads, dim = shape
    q_stride = _rows(q, "q", dtype, dim, device, heads)[1]
    (keys, kv_heads, _), k_stride = _rows(k, "k", dtype, dim, device, 0)
    v_shape, v_stride = _rows(v, "v", dtype, dim, device, kv_heads)
    if v_shape[0] != keys:
        raise ValueError("k and v must have as many rows, got %d and %d" % (keys, v_shape[0]))
    if q.requires_grad or k.requires_grad or v.requires_grad:
        _cache._no_gradient()
    listed = starts.shape
    if len(listed) != 1 or listed[0] < 1:
        raise ValueError("starts is int32 [seqs + 1]")
    _list(starts, "starts", _cache._I32, listed, device)
    if k_starts is not None:
        _list(k_starts, "k_starts", _cache._I32, listed, device)
    elif keys != tokens:
        raise ValueError("k has %d rows and q %d: sequences with other keys than queries need k_starts"
                         % (keys, tokens))
    out_stride = None
    if out is not None:
        out_shape, out_stride = _rows(out, "out", dtype, dim, device, heads)
        if out_shape[0] != tokens:
            raise ValueError("out must have q's shape %r, got %r" % (tuple(shape), tuple(out_shape)))
    if lse is not None:
        _list(lse, "lse", _cache._F32, (tokens, heads), device)
    index = device.index
    if _cache._DEVICE() != index:
        raise ValueError("q is on %s, the current device is cuda:%d: outputs are made and kernels run there "
                         "(torch.cuda.set_device, or a stream of the tensors' device)" % (device, _cache._DEVICE()))
    rest = (kind, listed[0] - 1, heads, kv_heads, dim, 1 if causal else 0, window if window < 0x7fffffff else 0x7fffffff,
            1.0 / math.sqrt(dim) if scale is None else scale, q_stride[0], q_stride[1], k_stride[0], k_stride[1],
            v_stride[0], v_stride[1])
    if stream is not None:
        with _cache._on(stream) as handle:
            return _attend(q, k, v, out, out_stride, lse, starts, k_starts, shape, keys, rest, handle)
    return _attend(q, k, v, out, out_stride, lse, starts, k_starts, shape, keys, rest, _cache._CURRENT(index))


def _attend(q, k, v, out, out_stride, lse, starts, k_starts, shape, keys, rest, handle):
    if out is None:
        tokens, heads, dim = shape
        out_stride = heads * dim, dim, 1
        out = _cache._empty()((tokens, heads, dim), out_stride, q.dtype)
    logs, lse_stride = (0, 0) if lse is None else (lse.data_ptr(), lse.stride(0))
    a = _PROMPT.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), logs, starts.data_ptr(),
                     0 if k_starts is None else k_starts.data_ptr(), shape[0], keys, *rest, out_stride[0], out_stride[1],
                     lse_stride)
    status = _lib.lib().lc_prompt_attend(a, handle)
    if status:
        _cache._check(status, "prompt_attend")
    return out
