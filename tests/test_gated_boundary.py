"""Argument checks of the gated pair, its way back and the transposed weights, on the host (no GPU)."""

import ctypes

import pytest
import torch

import hadamard_rotated_int8_amd as cr
from hadamard_rotated_int8_amd import block as impl

WEIGHT = dict(q=4096, scale=8192, bias=0, n=64, k=128, type=cr.E8M0)
PAIR = dict(y=16384, ldy=64, y_dtype=cr.BF16, act=cr.ACT_SILU, kept_gate=0, kept_up=0, ldk=64)
PACKED = dict(q=4096, scale=4096, m=0, k=128, lds=64)
BACK = dict(dy=4096, gate=8192, up=12288, dgate=16384, dup=20480, m=0, n=64, lddy=64, ldk=64, ldd=64,
            dy_dtype=cr.F32, act=cr.ACT_GELU)


def _weight(**kw):
    return impl._FP8_WEIGHTS.pack(*{**WEIGHT, **kw}.values())


def _pair(gate={}, up={}, **kw):
    return _weight(**gate) + _weight(**up) + impl._GATED_TAIL.pack(*{**PAIR, **kw}.values())


def _packed(**kw):
    return impl._FP8_PACKED.pack(*{**PACKED, **kw}.values())


def _gated(m=0, **kw):
    return cr.lib().convrot_fp8_gated(_packed(m=m), _pair(**kw), None)


def _rows(m=0, **kw):
    return cr.lib().convrot_fp8_gated_rows(4096, cr.BF16, m, 128, 128, _pair(**kw), None)


@pytest.mark.parametrize("call", [_gated, _rows])
def test_gated_arguments(call):
    assert call() == cr.OK
    assert call(m=1, gate=dict(n=0), up=dict(n=0)) == cr.OK
    for kw, status in [
            (dict(gate=dict(n=32)), cr.ERR_SHAPE), (dict(up=dict(k=144)), cr.ERR_SHAPE), (dict(ldy=63), cr.ERR_SHAPE),
            (dict(y_dtype=cr.I32), cr.ERR_DTYPE), (dict(act=cr.ACT_NONE), cr.ERR_DTYPE), (dict(act=3), cr.ERR_DTYPE),
            (dict(up=dict(type=cr.F32)), cr.ERR_DTYPE), (dict(kept_gate=65536), cr.ERR_NULL),
            (dict(kept_up=65536), cr.ERR_NULL), (dict(kept_gate=65536, kept_up=32768, ldk=63), cr.ERR_SHAPE),
            (dict(kept_gate=65536, kept_up=65536), cr.ERR_UNSUPPORTED),
            (dict(kept_gate=16384, kept_up=65536), cr.ERR_UNSUPPORTED),
            (dict(kept_gate=65536, kept_up=32769), cr.ERR_UNSUPPORTED),
            (dict(m=-1), cr.ERR_SHAPE), (dict(m=1, y=0), cr.ERR_NULL), (dict(m=1, gate=dict(q=0)), cr.ERR_NULL),
            (dict(m=1, up=dict(scale=0)), cr.ERR_NULL), (dict(m=1, up=dict(q=4100)), cr.ERR_UNSUPPORTED),
            (dict(m=1, y=16385), cr.ERR_UNSUPPORTED), (dict(m=1, gate=dict(bias=2)), cr.ERR_UNSUPPORTED)]:
        assert call(**kw) == status, kw


def test_gated_pointers():
    lib = cr.lib()
    assert lib.convrot_fp8_gated(None, _pair(), None) == cr.ERR_NULL
    assert lib.convrot_fp8_gated(_packed(), None, None) == cr.ERR_NULL
    assert lib.convrot_fp8_gated(_packed(m=1, lds=3), _pair(), None) == cr.ERR_UNSUPPORTED
    assert lib.convrot_fp8_gated(_packed(m=1, q=0), _pair(), None) == cr.ERR_NULL
    assert lib.convrot_fp8_gated_rows(4096, cr.BF16, 17, 128, 128, _pair(), None) == cr.ERR_SHAPE
    assert lib.convrot_fp8_gated_rows(4096, cr.BF16, 1, 128, 127, _pair(), None) == cr.ERR_SHAPE
    assert lib.convrot_fp8_gated_rows(4096, 9, 1, 128, 128, _pair(), None) == cr.ERR_DTYPE
    assert lib.convrot_fp8_gated_rows(0, cr.F32, 1, 128, 128, _pair(), None) == cr.ERR_NULL
    assert lib.convrot_fp8_gated_rows(4100, cr.F32, 1, 128, 128, _pair(), None) == cr.ERR_UNSUPPORTED


def _backward(lds=64, q=4096, **kw):
    pk = impl._writable(_packed(lds=lds, q=q))
    v = {**BACK, **kw}
    at = list(v.values())
    return cr.lib().convrot_fp8_gated_backward(impl._GATED_BACKWARD.pack(*at[:5], ctypes.addressof(pk), *at[5:]),
                                               None), pk


@pytest.mark.parametrize("kw, status", [
    (dict(m=-1), cr.ERR_SHAPE), (dict(n=0), cr.ERR_SHAPE), (dict(n=66600, lddy=66600, ldk=66600, ldd=66600), cr.ERR_SHAPE),
    (dict(lddy=63), cr.ERR_SHAPE), (dict(ldk=63), cr.ERR_SHAPE), (dict(ldd=63), cr.ERR_SHAPE),
    (dict(dy_dtype=cr.I32), cr.ERR_DTYPE), (dict(act=cr.ACT_NONE), cr.ERR_DTYPE), (dict(m=65), cr.ERR_SHAPE),
    (dict(m=1, lds=6), cr.ERR_UNSUPPORTED), (dict(m=1, q=0), cr.ERR_NULL), (dict(m=1, dy=0), cr.ERR_NULL),
    (dict(m=1, up=0), cr.ERR_NULL), (dict(m=1, dup=0), cr.ERR_NULL), (dict(m=1, dy=4098), cr.ERR_UNSUPPORTED),
    (dict(m=1, dgate=20480), cr.ERR_UNSUPPORTED), (dict(m=1, dgate=8192), cr.ERR_UNSUPPORTED),
    (dict(m=1, dup=4096), cr.ERR_UNSUPPORTED)])
def test_backward_arguments(kw, status):
    assert _backward(**kw)[0] == status
    assert cr.lib().convrot_fp8_gated_backward(None, None) == cr.ERR_NULL


def test_backward_sets_the_activations_sizes():
    st, pk = _backward(n=130, lddy=130, ldk=130, ldd=130)
    assert st == cr.OK
    assert impl._FP8_PACKED.unpack(pk.raw)[2:4] == (0, 512)


@pytest.mark.parametrize("ws, count, out, status", [
    ([{}], 0, 4096, cr.ERR_SHAPE), ([{}], 9, 4096, cr.ERR_SHAPE), ([dict(k=120)], 1, 4096, cr.ERR_UNSUPPORTED),
    ([{}, dict(k=144)], 2, 4096, cr.ERR_SHAPE), ([{}, dict(n=0)], 2, 4096, cr.ERR_SHAPE),
    ([{}, dict(type=cr.F32)], 2, 4096, cr.ERR_DTYPE), ([dict(type=cr.I32)], 1, 4096, cr.ERR_DTYPE),
    ([dict(q=0)], 1, 4096, cr.ERR_NULL), ([dict(scale=0)], 1, 4096, cr.ERR_NULL), ([{}], 1, 0, cr.ERR_NULL),
    ([{}], 1, 4100, cr.ERR_UNSUPPORTED), ([dict(n=100000), dict(n=50000)], 2, 4096, cr.ERR_SHAPE)])
def test_transpose_arguments(ws, count, out, status):
    args = b"".join(_weight(**w) for w in ws) + bytes(impl._FP8_WEIGHTS.size * 8)
    assert cr.lib().convrot_fp8_transpose_weights(args, count, out, 8192, None) == status
    assert cr.lib().convrot_fp8_transpose_weights(None, 1, out, 8192, None) == cr.ERR_NULL


def test_host_tensors_are_refused():
    w = cr.Fp8Weights(torch.zeros(16, 16, dtype=torch.float8_e4m3fn), torch.ones(1, 1))
    with pytest.raises(ValueError, match="device"):
        cr.fp8_gated(torch.zeros(1, 16), w, w)
    with pytest.raises(ValueError, match="device"):
        cr.fp8_gated_backward(torch.zeros(1, 16), (torch.zeros(1, 16),) * 2, w)
    with pytest.raises(ValueError, match="device"):
        cr.fp8_transpose_weights([w])
