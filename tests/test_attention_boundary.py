"""Attention's argument checks, on the host (no GPU)."""

import ctypes

import pytest
import torch

import hadamard_rotated_int8_amd as cr
from hadamard_rotated_int8_amd.attention import _ATTENTION

FIELDS = ("q k v out qb qt qh kb kt kh vb vt vh ob ot oh batch m l heads kv_heads d scale lengths mask "
          "mask_stride workspace workspace_bytes").split()
GOOD = dict(q=4096, k=8192, v=16384, out=32768, qb=6400, qt=640, qh=64, kb=6400, kt=640, kh=64, vb=6400,
            vt=640, vh=64, ob=6400, ot=640, oh=64, batch=1, m=0, l=10, heads=10, kv_heads=10, d=64,
            scale=0.125, lengths=0, mask=0, mask_stride=0, workspace=0, workspace_bytes=0)


def _apply(**kw):
    return cr.lib().convrot_attention_apply(_ATTENTION.pack(*[{**GOOD, **kw}[f] for f in FIELDS]), None)


def test_an_empty_call_is_no_error():
    assert _apply() == cr.OK
    assert _apply(m=5, batch=0) == cr.OK


@pytest.mark.parametrize("kw", [
    dict(batch=-1), dict(m=-1), dict(l=-1), dict(l=2 ** 31), dict(m=2 ** 31), dict(heads=0), dict(kv_heads=0),
    dict(heads=10, kv_heads=4), dict(heads=4097, kv_heads=1), dict(d=0), dict(d=200), dict(d=-8),
    dict(m=2 ** 30, heads=10, kv_heads=2), dict(m=2 ** 30, batch=2 ** 10),
    dict(m=1, qt=-8), dict(m=1, kt=56), dict(m=1, vt=8), dict(m=1, oh=2 ** 41), dict(m=1, kt=2 ** 24), dict(m=1, vt=2 ** 24),
    dict(mask=64, mask_stride=-1)])
def test_shapes_are_refused(kw):
    assert _apply(**kw) == cr.ERR_SHAPE


@pytest.mark.parametrize("kw", [
    dict(d=60), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
    dict(m=1, qt=644), dict(m=1, kh=4), dict(m=1, vb=1), dict(m=1, q=4100), dict(m=1, out=32770),
    dict(m=1, k=8194), dict(m=1, lengths=2), dict(m=1, out=4096), dict(m=1, out=16384)])
def test_unsupported_arguments_are_refused(kw):
    assert _apply(**kw) == cr.ERR_UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(q=0), dict(k=0), dict(v=0), dict(out=0)])
def test_missing_tensors_are_refused(kw):
    assert _apply(m=1, **kw) == cr.ERR_NULL
    assert cr.lib().convrot_attention_apply(None, None) == cr.ERR_NULL


def test_the_workspace_call_checks_its_arguments():
    need = ctypes.c_int64(-1)
    pack = lambda **kw: _ATTENTION.pack(*[{**GOOD, **kw}[f] for f in FIELDS])  # noqa: E731
    fn = cr.lib().convrot_attention_workspace
    assert fn(None, ctypes.byref(need)) == cr.ERR_NULL
    assert fn(pack(), None) == cr.ERR_NULL
    assert fn(pack(d=200), ctypes.byref(need)) == cr.ERR_SHAPE
    assert fn(pack(d=60), ctypes.byref(need)) == cr.ERR_UNSUPPORTED
    assert need.value == -1
    assert fn(pack(m=0), ctypes.byref(need)) == cr.OK and need.value == 0


def test_host_tensors_are_refused():
    q = torch.zeros(2, 3, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device"):
        cr.attention(q, q, q)
