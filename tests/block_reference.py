"""Plain 64-bit implementations of the operators around a block's linears, on the CPU.

Written from the definitions in include/convrot.h; the tests compare the HIP
kernels with these and with nothing else.
"""

import math

import torch

BLOCK = 128


def e4m3_nearest(v):
    """v (float64) to the nearest E4M3 value, ties to even (|v| <= 448)."""
    mag = v.abs()
    exponent = torch.frexp(mag.clamp_min(2.0 ** -6)).exponent - 1  # mag in [2^e, 2^(e+1))
    step = torch.ldexp(torch.ones_like(v), exponent - 3)
    return torch.round(v / step) * step


def block_scale(top):
    """The power of two (float64) of a block with largest magnitude `top`, and its E8M0 byte."""
    f = torch.frexp(top / 448)
    e = torch.where(f.mantissa == 0.5, f.exponent - 1, f.exponent).clamp(-126, 127)
    e = torch.where(top == 0, torch.zeros_like(e), e)
    bad = ~torch.isfinite(top)
    byte = torch.where(bad, torch.full_like(e, 255), e + 127)
    s = torch.where(bad, torch.full_like(top, math.nan), torch.ldexp(torch.ones_like(top), e.clamp(-300, 300)))
    return s, byte


def pack(x):
    """(dequantised float64 [m, k], E8M0 bytes [m, kb]) of activations in blocks of 1 x 128."""
    x = x.double()
    m, k = x.shape
    kb = -(-k // BLOCK)
    b = torch.zeros(m, kb * BLOCK, dtype=torch.float64)
    b[:, :k] = x
    b = b.view(m, kb, BLOCK)
    top = torch.where(torch.isnan(b), math.inf, b).abs().amax(2)
    s, byte = block_scale(top)
    d = torch.where(torch.isnan(s)[..., None], math.nan, e4m3_nearest(b / s[..., None]) * s[..., None])
    return d.view(m, -1)[:, :k], byte


def quantize(w):
    """(dequantised float64 [n, k], E8M0 bytes [nb, kb]) of weights in blocks of 128 x 128."""
    w = w.double()
    n, k = w.shape
    nb, kb = -(-n // BLOCK), -(-k // BLOCK)
    b = torch.zeros(nb * BLOCK, kb * BLOCK, dtype=torch.float64)
    b[:n, :k] = w
    b = b.view(nb, BLOCK, kb, BLOCK)
    top = torch.where(torch.isnan(b), math.inf, b).abs().amax((1, 3))
    s, byte = block_scale(top)
    s = s[:, None, :, None]
    d = torch.where(torch.isnan(s), math.nan, e4m3_nearest(b / s) * s)
    return d.reshape(nb * BLOCK, kb * BLOCK)[:n, :k], byte


def codes(q):
    """E4M3 codes as float64 values."""
    return q.cpu().float().double()


def dequantised_rows(q, scale):
    k = q.shape[1]
    return codes(q) * scale.cpu().float().double().repeat_interleave(BLOCK, 1)[:, :k]


def dequantised_weights(q, scale):
    n, k = q.shape
    s = scale.cpu().float().double().repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]
    return codes(q) * s


def gelu(y):
    return y * torch.special.ndtr(y)


def norm(v, kind, eps, weight=None, bias=None):
    v = v.double()
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    v = v / torch.sqrt((v * v).mean(1, keepdim=True) + eps)
    if weight is not None:
        v = v * weight.cpu().double()
    if bias is not None:
        v = v + bias.cpu().double()
    return v


def rows_of(v, m):
    """A [k] or [groups, k] vector as one row for each of m rows (float64)."""
    v = v.cpu().double()
    v = v[None] if v.dim() == 1 else v
    return v.repeat_interleave(m // v.shape[0], 0)


def block(x, branch=None, gate=None, residual_scale=1.0, post=None, pre=None, scale=None, shift=None):
    """(h, y) in float64; post and pre are (kind, eps, weight, bias) or None."""
    m = x.shape[0]
    h = x.cpu().double()
    if branch is not None:
        b = branch.cpu().double()
        if post is not None:
            b = norm(b, *post)
        if gate is not None:
            b = b * rows_of(gate, m)
        h = residual_scale * h + b
    y = h if pre is None else norm(h, *pre)
    if scale is not None:
        y = y * (1 + rows_of(scale, m))
    if shift is not None:
        y = y + rows_of(shift, m)
    return h, y


def rope(x, inv_freq, layout, positions, axis=None, factor=1.0, start=0, inverse=False):
    """x [batch, tokens, heads, d] (or without batch) turned, in float64."""
    x = x.cpu().double()
    p = positions.cpu().double()
    inv_freq = inv_freq.cpu()
    rot = 2 * inv_freq.numel()
    if axis is None:
        angle = p[..., None] * inv_freq
    else:
        angle = p[..., axis.cpu().long()] * inv_freq  # [.., tokens, pairs]
    if x.dim() == 4 and angle.dim() == 2:
        angle = angle[None]
    angle = angle.unsqueeze(-2)  # heads
    c, s = angle.cos() * factor, angle.sin() * factor
    if inverse:
        s = -s
    out = x.clone()
    part = x[..., start:start + rot]
    if layout == "half":
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        out[..., start:start + rot] = torch.cat([a * c - b * s, b * c + a * s], -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        out[..., start:start + rot] = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    return out
