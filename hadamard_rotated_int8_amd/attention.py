"""Attention to an encoder's states, or of tokens to one another.

Argument checks and marshalling only, like the package's other helpers.
"""

from __future__ import annotations

import struct

import torch

from . import lib
from .block import _DETACH, _device, _launch, _no_gradient, _no_overlap, _recording, _span, _workspace

MAX_HEAD_DIM = 192

_ATTENTION = struct.Struct("=4Q12q3q3ifQQqQq")


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, scale: float | None = None,
              lengths: torch.Tensor | None = None, mask: torch.Tensor | None = None,
              out: torch.Tensor | None = None) -> torch.Tensor:
    """softmax(scale q k^T) v of each head, in one pass over the keys.

    q       : bfloat16 [batch, m, heads, d] or [m, heads, d]
    k, v    : bfloat16 [batch, l, kv_heads, d] or [l, kv_heads, d]; kv_heads divides heads, and
              query head h reads key head h // (heads // kv_heads)
    scale   : 1 / sqrt(d) by default
    lengths : int32 [batch]: a batch entry's keys from there on are hidden
    mask    : bool [batch, l] or [l]: the keys that are seen
    out     : where the result goes, in memory of its own; by default a new contiguous tensor
    d is a multiple of 8 up to 192.  Any strides but 1 along d that are multiples of 8, 16-byte
    aligned (column ranges of a projection's rows, expanded batches).  Returns bfloat16 in q's
    shape; a query that sees no key gives zeros.  Hidden keys and values may hold anything.  There is
    no gradient: autograd raises where it comes back to the result.
    """
    dev = _device(q, "q")
    if _recording() and (q.requires_grad or k.requires_grad or v.requires_grad):
        return _no_gradient(attention, (q, k, v, scale, lengths, mask), _DETACH, out, q, k, v)
    dim = q.dim()
    known = dim == 3 or dim == 4
    for t, what in ((q, "q"), (k, "k"), (v, "v")):
        if not known or t.dtype != torch.bfloat16 or t.dim() != dim or (t.stride(-1) != 1 and t.shape[-1] != 1):
            raise ValueError(f"{what} must be bfloat16 [batch, tokens, heads, d] or [tokens, heads, d] "
                             "with unit stride along d")
        if t.device != dev:
            raise ValueError("all tensors of one call must be on the same device")
    m, heads, d = q.shape[-3:]
    l, kv_heads = k.shape[-3:-1]
    batch = q.shape[0] if dim == 4 else 1
    if k.shape != v.shape or k.shape[-1] != d or (dim == 4 and k.shape[0] != batch):
        raise ValueError("k and v must share one shape, and q's batch and d")
    if kv_heads < 1 or heads < 1 or heads % kv_heads:
        raise ValueError("the heads of k must divide those of q")
    if lengths is not None:
        if lengths.dtype != torch.int32 or lengths.shape != (batch,) or not lengths.is_contiguous():
            raise ValueError("lengths must be a contiguous int32 [batch] tensor")
        if lengths.device != dev:
            raise ValueError("all tensors of one call must be on the same device")
    mask_stride = 0
    if mask is not None:
        if mask.dtype != torch.bool or mask.shape not in ((l,), (batch, l)) or \
                (mask.stride(-1) != 1 and l != 1):
            raise ValueError("mask must be bool [batch, l] or [l] with unit stride along the keys")
        if mask.device != dev:
            raise ValueError("all tensors of one call must be on the same device")
        mask_stride = mask.stride(0) if mask.dim() == 2 else 0
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        if out.dtype != torch.bfloat16 or out.shape != q.shape or out.stride(-1) != 1 or out.device != dev:
            raise ValueError("out must be bfloat16 of q's shape and device with unit stride along d")
        if not _no_overlap(out):
            raise ValueError("out's elements must not overlap")
        lo, hi = _span(out)
        if any(a < hi and lo < b for a, b in map(_span, [t for t in (q, k, v, lengths, mask) if t is not None])):
            raise ValueError("out must not lie over an input")

    def strides(t):
        st = t.stride()[:3] if dim == 4 else (0, *t.stride()[:2])
        if (st[0] | st[1] | st[2]) & 7:  # (an axis of one may state any distance)
            st = tuple(0 if n == 1 else s for s, n in zip(st, t.shape[:3] if dim == 4 else (1, *t.shape[:2])))
        return st

    if scale is None:
        scale = d ** -0.5 if d else 1.0
    args = [q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), *strides(q), *strides(k),
            *strides(v), *strides(out), batch, m, l, heads, kv_heads, d, scale,
            0 if lengths is None else lengths.data_ptr(), 0 if mask is None else mask.data_ptr(),
            mask_stride, 0, 0]
    packed, space = _workspace(lib().convrot_attention_workspace, "convrot_attention_workspace", args,
                               _ATTENTION, dev, (batch, m, l, heads, kv_heads, d))
    _launch(lib().convrot_attention_apply, "convrot_attention_apply", dev, packed)
    return out
