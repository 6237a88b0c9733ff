"""The group norm's argument checks, on the host (no GPU)."""

import ctypes

import pytest
import torch

import hadamard_rotated_int8_amd as cr
from hadamard_rotated_int8_amd.block import _GROUP_NORM

FIELDS = ("x y xb xp yb yp batch positions c groups x_dtype y_dtype eps silu w ws wr wt b bs br bt "
          "workspace workspace_bytes").split()
GOOD = dict(x=4096, y=8192, xb=640, xp=64, yb=640, yp=64, batch=1, positions=0, c=64, groups=8, x_dtype=cr.F32,
            y_dtype=cr.BF16, eps=1e-6, silu=1, w=0, ws=0, wr=1, wt=0, b=0, bs=0, br=1, bt=0, workspace=0,
            workspace_bytes=0)


def _pack(**kw):
    return _GROUP_NORM.pack(*[{**GOOD, **kw}[f] for f in FIELDS])


def _apply(**kw):
    return cr.lib().convrot_group_norm_apply(_pack(**kw), None)


def test_an_empty_call_is_no_error():
    assert _apply() == cr.OK
    assert _apply(batch=0, positions=9) == cr.OK


@pytest.mark.parametrize("kw, status", [
    (dict(batch=-1), cr.ERR_SHAPE), (dict(positions=-1), cr.ERR_SHAPE), (dict(positions=2 ** 31), cr.ERR_SHAPE),
    (dict(c=0), cr.ERR_SHAPE), (dict(c=4104), cr.ERR_SHAPE), (dict(groups=0), cr.ERR_SHAPE),
    (dict(groups=7), cr.ERR_SHAPE), (dict(groups=-8), cr.ERR_SHAPE), (dict(xb=-1), cr.ERR_SHAPE),
    (dict(yp=2 ** 41), cr.ERR_SHAPE), (dict(x_dtype=cr.I32), cr.ERR_DTYPE), (dict(y_dtype=7), cr.ERR_DTYPE),
    (dict(silu=2), cr.ERR_DTYPE), (dict(eps=-1.0), cr.ERR_UNSUPPORTED), (dict(eps=float("nan")), cr.ERR_UNSUPPORTED),
    (dict(w=64, wt=9), cr.ERR_DTYPE), (dict(b=2), cr.ERR_UNSUPPORTED),
    (dict(positions=1, x=0), cr.ERR_NULL), (dict(positions=1, y=0), cr.ERR_NULL),
    (dict(positions=1, x=4098), cr.ERR_UNSUPPORTED), (dict(positions=1, y=4096), cr.ERR_UNSUPPORTED),
    (dict(positions=1, y=4096, y_dtype=cr.F32, yb=6400), cr.ERR_UNSUPPORTED)])
def test_bad_arguments_are_refused(kw, status):
    assert _apply(**kw) == status
    assert cr.lib().convrot_group_norm_apply(None, None) == cr.ERR_NULL


def test_the_workspace_call_checks_its_arguments():
    need = ctypes.c_int64(-1)
    fn = cr.lib().convrot_group_norm_workspace
    assert fn(None, ctypes.byref(need)) == cr.ERR_NULL
    assert fn(_pack(), None) == cr.ERR_NULL
    assert fn(_pack(groups=5), ctypes.byref(need)) == cr.ERR_SHAPE
    assert need.value == -1
    assert fn(_pack(positions=1024), ctypes.byref(need)) == cr.OK and need.value == 0  # in one workgroup


def test_host_tensors_are_refused():
    with pytest.raises(ValueError, match="device"):
        cr.group_norm(torch.zeros(1, 2, 8), 2)
