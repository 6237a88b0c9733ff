"""The operators around a transformer block's linears: FP8 linears with a scale
for each block of 128 features, the norms before and after a block with its
gate and residual, and rotary positions.

Argument checks and marshalling only, like the package's other helpers: every
step of the computation runs in the HIP kernels of libconvrot.so.  The call
path is kept short (arguments are packed straight into the C structs of
include/convrot.h), since a single token's operators cost a few microseconds
on the GPU.

``block_norm`` -> ``fp8_linear_grouped`` (Q, K, V) -> ``rope`` -> attention ->
``fp8_linear`` -> ``block_update`` -> ``fp8_linear`` (GELU) -> ``fp8_linear`` ->
``block_update`` is one block of a diffusion transformer; ``block_norm`` and
``block_update`` can hand the next linear its FP8 activation directly.
"""

from __future__ import annotations

import ctypes
import math
import struct
from dataclasses import dataclass

import torch

from . import ACT_GELU, ACT_NONE, BF16, E8M0, F32, MAX_GROUPED, OK, ConvrotError, lib

FP8_BLOCK = 128
FP8_MAX_ROWS, FP8_MAX_ROWS_BYTES = 16, 49152  # an activation that is quantised inside the linear
MAX_NORM_K = 32768
MAX_ROPE_TENSORS = 4

_DTYPE = {torch.float32: F32, torch.bfloat16: BF16}
_E8M0 = getattr(torch, "float8_e8m0fnu", None)  # (newer than the rest of what the package needs)
_SCALE_DTYPE = {torch.float32: F32, _E8M0: E8M0}
_POSITION = {torch.int32: 0, torch.int64: 1, torch.float32: 2}

# The structs of include/convrot.h, as struct formats.
_FP8_PACKED = struct.Struct("=QQqqq")
_FP8_WEIGHTS = struct.Struct("=QQQqqi4x")
_VECTOR = "Qqqi4x"
_NORM = "if" + _VECTOR + _VECTOR
_BLOCK = struct.Struct("=5Q6q3if" + 3 * _VECTOR + 2 * _NORM)
_ROPE_TENSOR = "QQ7q"
_ROPE = struct.Struct("=3Q4q8ifii4x" + 4 * _ROPE_TENSOR)

_ROPE_PADDING = [(0,) * 9 * (MAX_ROPE_TENSORS - i) for i in range(MAX_ROPE_TENSORS + 1)]

_ABSENT = (0, 0, 1, 0)
_NO_NORM = (0, 0.0, *_ABSENT, *_ABSENT)


def _writable(b: bytes):
    """A C buffer holding b that the library may write to."""
    return ctypes.create_string_buffer(b, len(b))


def _launch(fn, name, dev, *args):
    """fn(*args, stream) on dev's current stream, with dev the current device."""
    i = dev.index
    if torch._C._cuda_getDevice() == i:
        st = fn(*args, torch._C._cuda_getCurrentRawStream(i))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(i))
    if st != OK:
        raise ConvrotError(st, name)


def _device(x: torch.Tensor, what: str) -> torch.device:
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError(f"{what} must be a device tensor")
    return x.device


def _rows(x: torch.Tensor, what: str, dev=None, shape=None) -> int:
    """Check a float matrix with unit column stride; returns its type's code."""
    dt = _DTYPE.get(x.dtype)
    if dt is None or x.dim() != 2 or (x.stride(1) != 1 and x.shape[1] != 1):
        raise ValueError(f"{what} must be a float32 or bfloat16 matrix with unit column stride")
    if shape is not None and x.shape != shape:
        raise ValueError(f"{what} must have the shape {tuple(shape)}")
    if dev is not None and x.device != dev:
        raise ValueError("all tensors of one call must be on the same device")
    return dt


def _row_stride(x: torch.Tensor) -> int:
    """The row stride of a checked matrix (one row has any, down to its length)."""
    stride, k = x.stride(0), x.shape[1]
    return stride if stride >= k or x.shape[0] > 1 else k


def _writable_rows(x: torch.Tensor, what: str) -> None:
    if x.shape[0] > 1 and x.stride(0) < x.shape[1]:
        raise ValueError(f"the rows of {what} must not overlap")


def _new_like(x: torch.Tensor, dtype: torch.dtype, dev) -> torch.Tensor:
    """A contiguous tensor of x's shape (empty_like is the shorter call where it gives one)."""
    if dtype == x.dtype and x.is_contiguous():
        return torch.empty_like(x)
    return torch.empty(x.shape, dtype=dtype, device=dev)


def _span(x: torch.Tensor) -> tuple[int, int]:
    """The addresses from a matrix's first byte to behind its last."""
    at = x.data_ptr()
    if x.numel() == 0:
        return at, at
    return at, at + (1 + sum((n - 1) * s for n, s in zip(x.shape, x.stride()))) * x.element_size()


def _distinct(outs) -> None:
    at = [o.data_ptr() for o in outs if o.numel()]
    if len(set(at)) != len(at):
        raise ValueError("the outputs of one call must not overlap")


# ---------------------------------------------------------------------------
# FP8 linears
# ---------------------------------------------------------------------------

@dataclass
class Fp8Weights:
    """E4M3 [n, k] codes, one scale for each block of 128 x 128, optional float32 [n] bias.

    ``scale`` is [ceil(n / 128), ceil(k / 128)], float8_e8m0fnu (powers of two,
    what ``fp8_quantize_weights`` writes) or float32 (any scales, as
    checkpoints hold them).
    """

    q: torch.Tensor
    scale: torch.Tensor
    bias: torch.Tensor | None = None


@dataclass
class Fp8Activation:
    """E4M3 [m, k] codes and their E8M0 scales [m, ceil(k / 128)], one for each row and block.

    The scales lie block by block: stride 1 along the rows, a multiple of 4 along the blocks
    (``fp8_pack_activations`` pads it).  Rows from one multiple of 4 to another can be taken as
    ``Fp8Activation(p.q[a:b], p.scale[a:b])``.
    """

    q: torch.Tensor
    scale: torch.Tensor


def _blocks(n: int) -> int:
    return -(-n // FP8_BLOCK)


def _new_scales(*shape, device) -> torch.Tensor:
    if _E8M0 is None:
        raise RuntimeError("FP8 scales need a torch that has float8_e8m0fnu")
    return torch.empty(shape, dtype=_E8M0, device=device)


def _new_activation(m: int, k: int, dev) -> Fp8Activation:
    q = torch.empty((m, k), dtype=torch.float8_e4m3fn, device=dev)
    scale = _new_scales(_blocks(k), (m + 3) // 4 * 4, device=dev)
    return Fp8Activation(q, scale.t()[:m])


def _check_activation(x: Fp8Activation) -> torch.device:
    q, s = x.q, x.scale
    dev = _device(q, "the FP8 codes")
    if q.dtype != torch.float8_e4m3fn or q.dim() != 2 or not q.is_contiguous():
        raise ValueError("the FP8 codes must be a contiguous float8_e4m3fn [m, k] tensor")
    m, kb = q.shape[0], _blocks(q.shape[1])
    if s.dtype != _E8M0 or s.shape != (m, kb) or (s.stride(0) != 1 and m > 1):
        raise ValueError("the FP8 scales must be a float8_e8m0fnu [m, ceil(k / 128)] tensor with "
                         "unit row stride")
    if s.device != dev:
        raise ValueError("all tensors of one call must be on the same device")
    # whole words are read: the padding behind the last row has to be there
    if m and kb and s.storage_offset() + (kb - 1) * s.stride(1) + (m + 3) // 4 * 4 > \
            s.untyped_storage().nbytes():
        raise ValueError("the FP8 scales must be padded to a multiple of 4 rows")
    return dev


def _pack_args(x: Fp8Activation) -> bytes:
    m, k = x.q.shape
    s = x.scale
    # the distance of a single block says nothing: any that holds the rows will do
    lds = s.stride(1) if s.shape[1] > 1 else (m + 3) // 4 * 4
    return _FP8_PACKED.pack(x.q.data_ptr(), s.data_ptr(), m, k, lds)


def fp8_quantize_weights(w: torch.Tensor, bias: torch.Tensor | None = None) -> Fp8Weights:
    """E4M3 codes and E8M0 scales of W (float32 or bfloat16 [n, k]) in blocks of 128 x 128."""
    dev = _device(w, "w")
    dt = _rows(w, "w")
    n, k = w.shape
    _check_bias(bias, n, dev)
    q = torch.empty((n, k), dtype=torch.float8_e4m3fn, device=dev)
    scale = _new_scales(_blocks(n), _blocks(k), device=dev)
    _launch(lib().convrot_fp8_quantize_weights, "convrot_fp8_quantize_weights", dev, w.data_ptr(),
            dt, n, k, _row_stride(w), q.data_ptr(), scale.data_ptr())
    return Fp8Weights(q, scale, bias)


def fp8_pack_activations(x: torch.Tensor, out: Fp8Activation | None = None) -> Fp8Activation:
    """E4M3 codes and E8M0 scales of X in blocks of 1 x 128.

    x: float32 or bfloat16 [m, k], k a multiple of 16, rows at multiples of 16 bytes.
    """
    dev = _device(x, "x")
    dt = _rows(x, "x")
    m, k = x.shape
    if out is None:
        out = _new_activation(m, k, dev)
    elif _check_activation(out) != dev or out.q.shape != x.shape:
        raise ValueError("out must hold [m, k] codes on x's device")
    _launch(lib().convrot_fp8_pack_activations, "convrot_fp8_pack_activations", dev, x.data_ptr(),
            dt, m, k, _row_stride(x), _writable(_pack_args(out)))
    return out


def _check_bias(bias, n, dev):
    if bias is not None:
        if bias.dtype != torch.float32 or bias.shape != (n,) or not bias.is_contiguous():
            raise ValueError("bias must be a contiguous float32 [n] tensor")
        if bias.device != dev:
            raise ValueError("all tensors of one call must be on the same device")


def fp8_linear_grouped(x: torch.Tensor | Fp8Activation, ws, outs=None,
                       out_dtype: torch.dtype = torch.float32, gelu: bool = False):
    """Several FP8 linears on one activation in one launch; returns the outputs.

    x: float32 or bfloat16 [m, k], which is packed on the way, or what
    ``fp8_pack_activations``, ``block_norm`` or ``block_update`` packed.  k is a
    multiple of 16, and the rows of an unpacked x start at multiples of 16 bytes.
    How the sums are divided depends on the sizes of the whole call, so a row's
    last bits may differ between calls of different sizes (the same call gives
    the same bits).
    Output i is act(X W_i^T + bias_i), float32 or bfloat16 [m, n_i].  Sums are
    float32; for bfloat16 outputs products more than 13 bits below the largest
    of 8 neighbouring features are cut (include/convrot.h states the bound).
    ``outs`` may lie over an unpacked x, not over one another.
    """
    if not ws or len(ws) > MAX_GROUPED:
        raise ValueError(f"1 to {MAX_GROUPED} weights")
    rows = None
    if isinstance(x, Fp8Activation):
        dev = _check_activation(x)
        m, k = x.q.shape
    else:
        dev = _device(x, "x")
        rows = _rows(x, "x")
        m, k = x.shape
        if m > FP8_MAX_ROWS or m * _blocks(k) * FP8_BLOCK > FP8_MAX_ROWS_BYTES:
            x, rows = fp8_pack_activations(x), None
    dt = _DTYPE.get(out_dtype)
    if dt is None:
        raise ValueError("out_dtype must be torch.float32 or torch.bfloat16")
    packed = []
    for w in ws:
        q, s = w.q, w.scale
        if q.dtype != torch.float8_e4m3fn or q.dim() != 2 or not q.is_contiguous():
            raise ValueError("weight codes must be a contiguous float8_e4m3fn [n, k] tensor")
        n = q.shape[0]
        sdt = _SCALE_DTYPE.get(s.dtype)
        if sdt is None or s.shape != (_blocks(n), _blocks(q.shape[1])) or not s.is_contiguous():
            raise ValueError("weight scales must be a contiguous float8_e8m0fnu or float32 "
                             "[ceil(n / 128), ceil(k / 128)] tensor")
        b = w.bias
        _check_bias(b, n, dev)
        if q.device != dev or s.device != dev:
            raise ValueError("all tensors of one call must be on the same device")
        packed.append(_FP8_WEIGHTS.pack(q.data_ptr(), s.data_ptr(),
                                        0 if b is None else b.data_ptr(), n, q.shape[1], sdt))
    if outs is None:
        outs = [torch.empty((m, w.q.shape[0]), dtype=out_dtype, device=dev) for w in ws]
    else:
        if len(outs) != len(ws):
            raise ValueError("one output per weight")
        for o, w in zip(outs, ws):
            if o.dtype != out_dtype:
                raise ValueError("the outputs must be of out_dtype")
            _rows(o, "an output", dev, (m, w.q.shape[0]))
            _writable_rows(o, "an output")
        _distinct(outs)
        if rows is not None:  # a workgroup may write Y while another still reads X
            lo, hi = _span(x)
            if any(a < hi and lo < b for a, b in map(_span, outs)):
                x, rows = fp8_pack_activations(x), None
    count = len(ws)
    args = (b"".join(packed), count, struct.pack(f"={count}Q", *[o.data_ptr() for o in outs]),
            struct.pack(f"={count}q", *[_row_stride(o) for o in outs]), dt,
            ACT_GELU if gelu else ACT_NONE)
    if rows is None:
        _launch(lib().convrot_fp8_linear_grouped, "convrot_fp8_linear_grouped", dev, _pack_args(x), *args)
    else:
        _launch(lib().convrot_fp8_linear_rows, "convrot_fp8_linear_rows", dev, x.data_ptr(), rows, m, k,
                _row_stride(x), *args)
    return outs


def fp8_linear(x: torch.Tensor | Fp8Activation, w: Fp8Weights, out: torch.Tensor | None = None,
               out_dtype: torch.dtype | None = None, gelu: bool = False) -> torch.Tensor:
    """act(X W^T + bias) on one FP8 weight; see ``fp8_linear_grouped``."""
    if out_dtype is None:
        out_dtype = torch.float32 if out is None else out.dtype
    return fp8_linear_grouped(x, (w,), None if out is None else (out,), out_dtype, gelu)[0]


# ---------------------------------------------------------------------------
# Norms around a block
# ---------------------------------------------------------------------------

@dataclass
class Norm:
    """A norm over the features of a row: ``kind`` "layer" or "rms", with optional weight and bias [k]
    (float32 or bfloat16)."""

    kind: str
    eps: float = 1e-6
    weight: torch.Tensor | None = None
    bias: torch.Tensor | None = None


_NORM_KIND = {"layer": 1, "rms": 2}


def _vector_args(v, k: int, what: str, dev):
    if v is None:
        return _ABSENT
    dt = _DTYPE.get(v.dtype)
    if dt is None or v.shape != (k,) or (v.stride(0) != 1 and k != 1):
        raise ValueError(f"{what} must be a float32 or bfloat16 [k] tensor with unit stride")
    if v.device != dev:
        raise ValueError("all tensors of one call must be on the same device")
    return v.data_ptr(), 0, 1, dt


def _norm_args(n, k: int, what: str, dev):
    if n is None:
        return _NO_NORM
    kind = _NORM_KIND.get(n.kind)
    if kind is None:
        raise ValueError(f"{what}: a norm is \"layer\" or \"rms\"")
    return (kind, n.eps, *_vector_args(n.weight, k, f"{what}: weight", dev),
            *_vector_args(n.bias, k, f"{what}: bias", dev))


def _group_args(v, m: int, k: int, what: str, dev):
    """A [k] vector, or [groups, k] with groups dividing m, as a C struct."""
    if v is None:
        return _ABSENT
    dt = _DTYPE.get(v.dtype)
    if dt is None or v.dim() not in (1, 2) or v.shape[-1] != k or (v.stride(-1) != 1 and k != 1):
        raise ValueError(f"{what} must be float32 or bfloat16, [k] or [groups, k], with unit "
                         "column stride")
    if v.device != dev:
        raise ValueError("all tensors of one call must be on the same device")
    groups = v.shape[0] if v.dim() == 2 else 1
    if groups == 1:
        return v.data_ptr(), 0, max(m, 1), dt
    if groups == 0 or m % groups:
        raise ValueError(f"{what}: its rows must divide the rows of x")
    return v.data_ptr(), v.stride(0), max(m // groups, 1), dt


def _block_call(x, branch, gate, residual_scale, post, norm, scale, shift, h, y, packed, dev):
    m, k = x.shape
    pk = 0
    if packed is not None:
        pk = _writable(_pack_args(packed))
    args = _BLOCK.pack(
        x.data_ptr(), 0 if branch is None else branch.data_ptr(), 0 if h is None else h.data_ptr(),
        0 if y is None else y.data_ptr(), ctypes.addressof(pk) if pk else 0, m, k, _row_stride(x),
        0 if branch is None else _row_stride(branch), 0 if h is None else _row_stride(h),
        0 if y is None else _row_stride(y), _DTYPE[x.dtype],
        0 if branch is None else _DTYPE[branch.dtype], 0 if y is None else _DTYPE[y.dtype],
        residual_scale, *_group_args(gate, m, k, "gate", dev),
        *_group_args(scale, m, k, "scale", dev), *_group_args(shift, m, k, "shift", dev),
        *_norm_args(post, k, "post", dev),
        *_norm_args(norm, k, "norm", dev))
    _launch(lib().convrot_block_norm, "convrot_block_norm", dev, args)


def _out_rows(out, x, out_dtype, pack, dev):
    """The (y, packed) outputs of a norm: one of them, as asked."""
    if pack:
        if out is None:
            return None, _new_activation(x.shape[0], x.shape[1], dev)
        if not isinstance(out, Fp8Activation) or _check_activation(out) != dev or \
                out.q.shape != x.shape:
            raise ValueError("with pack, out must be an Fp8Activation of x's shape on x's device")
        return None, out
    if out is None:
        return _new_like(x, out_dtype or x.dtype, dev), None
    _rows(out, "out", dev, x.shape)
    _writable_rows(out, "out")
    if out_dtype is not None and out.dtype != out_dtype:
        raise ValueError("out must be of out_dtype")
    return out, None


def block_norm(x: torch.Tensor, norm: Norm | None, scale: torch.Tensor | None = None,
               shift: torch.Tensor | None = None, out=None, out_dtype: torch.dtype | None = None,
               pack: bool = False):
    """norm(x) * (1 + scale) + shift: what a block's linears read.

    x: float32 or bfloat16 [m, k].  scale and shift: [k], or [groups, k] with
    m / groups consecutive rows to each (one row for each image of a batch).
    Returns float32 or bfloat16 [m, k] (x's type by default; ``out`` may be x),
    or with ``pack`` the Fp8Activation of it (k a multiple of 16).
    """
    dev = _device(x, "x")
    _rows(x, "x")
    if not pack and out_dtype is not None and out_dtype not in _DTYPE:
        raise ValueError("out_dtype must be torch.float32 or torch.bfloat16")
    y, packed = _out_rows(out, x, out_dtype, pack, dev)
    _block_call(x, None, None, 1.0, None, norm, scale, shift, None, y, packed, dev)
    return packed if pack else y


def block_update(x: torch.Tensor, branch: torch.Tensor, gate: torch.Tensor | None = None,
                 residual_scale: float = 1.0, post: Norm | None = None, norm: Norm | None = None,
                 scale: torch.Tensor | None = None, shift: torch.Tensor | None = None,
                 out_h: torch.Tensor | None = None, out=None,
                 out_dtype: torch.dtype | None = None, pack: bool = False):
    """A block's output onto its residual stream, and the next block's input, in one pass:

        h = residual_scale * x + gate * post(branch)
        y = norm(h) * (1 + scale) + shift

    Returns (h, y).  h has x's type; ``out_h`` may be x (in place).  y is None
    unless a norm, a scale or a shift is given; it is computed from h before h
    is rounded, and is a matrix or, with ``pack``, an Fp8Activation as in
    ``block_norm``.
    """
    dev = _device(x, "x")
    _rows(x, "x")
    _rows(branch, "branch", dev, x.shape)
    if out_dtype is not None and out_dtype not in _DTYPE:
        raise ValueError("out_dtype must be torch.float32 or torch.bfloat16")
    if out_h is None:
        out_h = _new_like(x, x.dtype, dev)
    else:
        if out_h.dtype != x.dtype:
            raise ValueError("out_h must have x's type")
        _rows(out_h, "out_h", dev, x.shape)
        _writable_rows(out_h, "out_h")
    y = packed = None
    if norm is not None or scale is not None or shift is not None:
        y, packed = _out_rows(out, x, out_dtype, pack, dev)
    elif out is not None or pack:
        raise ValueError("out and pack need a norm, a scale or a shift")
    _block_call(x, branch, gate, residual_scale, post, norm, scale, shift, out_h, y, packed, dev)
    return out_h, (packed if pack else y)


# ---------------------------------------------------------------------------
# Rotary positions
# ---------------------------------------------------------------------------

@dataclass
class RopePlan:
    """How the heads turn: one frequency for each pair of features.

    inv_freq : float64 [rot / 2] on the device
    layout   : "interleaved" (features 2j and 2j + 1) or "half" (j and j + rot / 2)
    axis     : int32 [rot / 2] on the device, which of a token's positions each
               pair turns by (time, row, column, ...), or None with one position
    factor   : multiplies cos and sin (long-context scalings use it)
    start    : first feature of the rotated slice
    axes     : how many positions a token has (0: not stated)
    """

    inv_freq: torch.Tensor
    layout: str = "interleaved"
    axis: torch.Tensor | None = None
    factor: float = 1.0
    start: int = 0
    axes: int = 0


def rope_plan(rot: int, theta: float = 10000.0, layout: str = "interleaved", axes=None,
              scaling: dict | None = None, start: int = 0, device="cuda") -> RopePlan:
    """The plan of a model's configuration; make it once.

    rot     : features of a head that turn (even)
    axes    : with several positions per token, the features of each (even, summing to rot)
    scaling : None, or a dict with a "type" for contexts longer than trained on
              linear   factor                    positions divided by factor
              ntk      factor                    theta raised so that the slowest pair is slowed by factor
              yarn     factor, original_length, beta_fast (32), beta_slow (1), attention_factor
                       pairs that turn more than beta_fast times over the original length are
                       kept, those that turn less than beta_slow times are slowed by factor, with a
                       ramp between; cos and sin times 0.1 ln(factor) + 1 unless attention_factor
                       is given
              factors  factors [rot / 2], attention_factor (1)   each frequency divided by its own
    """
    if rot < 2 or rot % 2 or start < 0:
        raise ValueError("rot must be even and positive, start at least 0")
    if layout not in _LAYOUT:
        raise ValueError('layout must be "interleaved" or "half"')
    if not theta > 1:
        raise ValueError("theta must be above 1")
    parts = [rot] if axes is None else list(axes)
    if sum(parts) != rot or any(p < 2 or p % 2 for p in parts):
        raise ValueError("axes must be even and sum to rot")
    scaling = dict(scaling or {})
    kind = scaling.pop("type", None)
    factor = 1.0
    divide = scaling.pop("factor", 1.0) if kind in ("linear", "ntk", "yarn") else 1.0
    if not divide >= 1:
        raise ValueError("a scaling factor is at least 1")
    if kind in ("ntk", "yarn") and axes is not None:
        raise ValueError(f"{kind} scaling is for a single position per token")
    if kind == "ntk" and rot > 2:
        theta *= divide ** (rot / (rot - 2))
    freqs = [theta ** (-2.0 * j / n) for n in parts for j in range(n // 2)]
    if kind == "linear":
        freqs = [f / divide for f in freqs]
    elif kind == "yarn":
        length = scaling.pop("original_length")
        fast, slow = scaling.pop("beta_fast", 32.0), scaling.pop("beta_slow", 1.0)
        if not (length > 0 and fast >= slow > 0):
            raise ValueError("yarn needs original_length > 0 and beta_fast >= beta_slow > 0")
        factor = scaling.pop("attention_factor", 0.1 * math.log(divide) + 1.0)

        def pair_of(turns):  # the pair that makes so many turns over the original length
            return rot * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(theta))

        low = max(math.floor(pair_of(fast)), 0)
        high = min(math.ceil(pair_of(slow)), rot - 1)
        ramp = [min(max((j - low) / max(high - low, 1e-3), 0.0), 1.0) for j in range(rot // 2)]
        freqs = [f * (1 - r) + f / divide * r for f, r in zip(freqs, ramp)]
    elif kind == "factors":
        each = [float(f) for f in scaling.pop("factors")]
        if len(each) != rot // 2 or not all(f > 0 for f in each):
            raise ValueError("factors must be rot / 2 positive numbers")
        factor = scaling.pop("attention_factor", 1.0)
        freqs = [f / d for f, d in zip(freqs, each)]
    elif kind not in (None, "ntk"):
        raise ValueError(f"unknown scaling type {kind!r}")
    if scaling:
        raise ValueError(f"unknown scaling keys {sorted(scaling)}")
    axis = None
    if axes is not None:
        axis = torch.tensor([i for i, n in enumerate(parts) for _ in range(n // 2)],
                            dtype=torch.int32, device=device)
    return RopePlan(torch.tensor(freqs, dtype=torch.float64, device=device), layout, axis,
                    float(factor), start, len(parts))


_LAYOUT = {"interleaved": 0, "half": 1}


def _no_overlap(x: torch.Tensor) -> bool:
    """Whether every element of x has a place of its own (sizes of one aside, strides that nest)."""
    reach = 1
    for stride, size in sorted((st, n) for st, n in zip(x.stride(), x.shape) if n > 1):
        if stride < reach:
            return False
        reach = stride * (size - 1) + reach
    return True


def rope(x, plan: RopePlan, positions: torch.Tensor, out=None, out_dtype: torch.dtype | None = None,
         inverse: bool = False):
    """Turn the heads of x, a tensor or a list of them (Q and K), in one launch.

    x         : float32 or bfloat16 [tokens, heads, d] or [batch, tokens, heads, d], any strides but 1
                along d; the tensors of a list share all but their heads and strides
    positions : int32, int64 or float32 [tokens] or [batch, tokens], with one more axis at the end
                where the plan has axes
    out       : where the results go (x itself turns in place); by default new tensors of
                out_dtype (x's type by default), contiguous
    inverse   : turn back
    """
    many = isinstance(x, (list, tuple))
    xs = x if many else (x,)
    count = len(xs)
    if not 1 <= count <= MAX_ROPE_TENSORS:
        raise ValueError(f"1 to {MAX_ROPE_TENSORS} tensors")
    first = xs[0]
    dev = _device(first, "x")
    dtype = first.dtype
    xdt = _DTYPE.get(dtype)
    if out is None:
        odt = dtype if out_dtype is None else out_dtype
        outs = [_new_like(t, odt, dev) for t in xs]
    else:
        outs = list(out) if many else [out]
        if len(outs) != count:
            raise ValueError("one output per tensor")
        _distinct(outs)
        odt = outs[0].dtype
        if out_dtype is not None and odt != out_dtype:
            raise ValueError("out must be of out_dtype")
    ydt = _DTYPE.get(odt)
    if xdt is None or ydt is None:
        raise ValueError("x and out must be float32 or bfloat16")
    inv, axis = plan.inv_freq, plan.axis
    layout = _LAYOUT.get(plan.layout)
    if layout is None:
        raise ValueError('layout must be "interleaved" or "half"')
    if inv.dtype != torch.float64 or inv.dim() != 1 or not inv.is_contiguous() or inv.device != dev:
        raise ValueError("inv_freq must be a contiguous float64 [rot / 2] tensor on x's device")
    rot = 2 * inv.shape[0]
    if axis is not None and (axis.dtype != torch.int32 or axis.shape != inv.shape or
                             not axis.is_contiguous() or axis.device != dev):
        raise ValueError("axis must be a contiguous int32 [rot / 2] tensor on x's device")
    dim = first.dim()
    if dim not in (3, 4):
        raise ValueError("x must be [tokens, heads, d] or [batch, tokens, heads, d]")
    batch = first.shape[0] if dim == 4 else 1
    tokens, _, d = first.shape[-3:]
    args = []
    for t, o in zip(xs, outs):
        shape, st = t.shape, t.stride()
        if len(shape) != dim or shape[-3] != tokens or shape[-1] != d or shape[0] != first.shape[0] or \
                t.dtype != dtype or t.device != dev or (st[-1] != 1 and d != 1):
            raise ValueError("the tensors must share type, device, batch, tokens and d, with unit "
                             "stride along d")
        to = o.stride()
        if out is not None:
            if o.shape != shape or o.dtype != odt or o.device != dev or to[-1] != 1:
                raise ValueError("an output must have its tensor's shape, with unit stride along d")
            if not _no_overlap(o):
                raise ValueError("an output's elements must not overlap")
            if o.data_ptr() == t.data_ptr() and (to != st or xdt != ydt):
                raise ValueError("in place, out must be x itself")
        if dim == 4:
            args += (t.data_ptr(), o.data_ptr(), *st[:3], *to[:3], shape[2])
        else:
            args += (t.data_ptr(), o.data_ptr(), 0, st[0], st[1], 0, to[0], to[1], shape[1])
    pdt = _POSITION.get(positions.dtype)
    lead = positions.dim() - (axis is not None)
    if pdt is None or positions.device != dev or lead not in (1, 2) or \
            positions.shape[lead - 1] != tokens or (lead == 2 and positions.shape[0] != batch):
        raise ValueError("positions must be int32, int64 or float32 [tokens] or [batch, tokens] "
                         "(with the plan's axes behind) on x's device")
    axes = 1
    if axis is not None:
        axes = positions.shape[-1]
        if axes < max(plan.axes, 1):
            raise ValueError("positions has fewer axes than the plan")
        if positions.stride(-1) != 1 and axes != 1:
            raise ValueError("the axes of a token's position must be consecutive")
    ps = positions.stride()
    _launch(lib().convrot_rope_apply, "convrot_rope_apply", dev,
            _ROPE.pack(inv.data_ptr(), 0 if axis is None else axis.data_ptr(), positions.data_ptr(),
                       ps[0] if lead == 2 else 0, ps[lead - 1], batch, tokens, pdt, d, rot,
                       plan.start, layout, 1 if inverse else 0, xdt, ydt, plan.factor, count, axes,
                       *args, *_ROPE_PADDING[count]))
    return outs if many else outs[0]
