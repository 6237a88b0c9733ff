"""Attention in 64 bits, and how far a float32 sum of bfloat16 weights may be from it."""

import torch


def seen_keys(batch, l, lengths=None, mask=None):
    """bool [batch, l]"""
    seen = torch.ones(batch, l, dtype=torch.bool)
    if lengths is not None:
        seen &= torch.arange(l) < lengths.cpu()[:, None]
    if mask is not None:
        seen &= mask.cpu()
    return seen


def attention_ref(q, k, v, scale=None, lengths=None, mask=None):
    """(out, tol) in float64 on the CPU for 4-dimensional bfloat16 inputs.

    With weights p_j (1 + a) rounded to bfloat16, |a| <= 2^-8, in the sum and at most in its divisor,
    and A = sum p |v| / sum p, the quotient is off by (2^-8 (A + |out|)) / (1 - 2^-8), and the output's own
    rounding by 2^-8 |out|.  A score's float32 sum of d products is off by (d + 1) 2^-24 sum |q k|,
    which the exponent carries, times scale, into a relative error of p; forming the exponent adds
    2^-22 of its size and the exponential 2^-22; the sums over l keys (l + 4) 2^-23 of A, twice (the
    weights' sum too).
    """
    batch, m, heads, d = q.shape
    l, kv = k.shape[1:3]
    scale = d ** -0.5 if scale is None else scale
    ratio = heads // kv
    seen = seen_keys(batch, l, lengths, mask)
    out = torch.zeros(batch, m, heads, d, dtype=torch.float64)
    tol = torch.zeros_like(out)
    q, k, v = (t.cpu().double() for t in (q, k, v))
    for b in range(batch):
        at = seen[b].nonzero()[:, 0]
        if at.numel() == 0:
            continue
        for h in range(heads):
            kk, vv, qq = k[b, at, h // ratio], v[b, at, h // ratio], q[b, :, h]
            s = qq @ kk.t() * scale
            top = s.amax(dim=1, keepdim=True)
            p = torch.exp(s - top)
            total = p.sum(dim=1, keepdim=True)
            o = p @ vv / total
            size = p @ vv.abs() / total
            err_s = (qq.abs() @ kk.abs().t() * scale * (d + 1) * 2 ** -24).amax(dim=1, keepdim=True)
            err_s = 2 * err_s + (top - s).amax(dim=1, keepdim=True) * 2 ** -21 + 2 ** -21
            out[b, :, h] = o
            tol[b, :, h] = (1.01 * 2 ** -8 * (size + 2 * o.abs())
                            + (size + o.abs()) * (err_s + (l + 4) * 2 ** -22) + 1e-30)
    return out, tol
