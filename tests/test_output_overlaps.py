"""Refusals of outputs over what other workgroups still read: on the host with made-up addresses, and through
the Python entry points (GPU)."""

import pytest
import torch

import hadamard_rotated_int8_amd as cr
import test_gated_boundary as gated
import test_group_norm_boundary as group_norm
from test_block_boundary import cpu_only

F32, BF16 = torch.float32, torch.bfloat16


# y: [2, 3, 64] bfloat16 from 8192 on, images 640 and positions 64 values apart: bytes 8192 .. 9855
@cpu_only
@pytest.mark.parametrize("kw", [dict(w=8192), dict(b=8192), dict(w=9852), dict(b=9852), dict(w=8192 - 252),
                                dict(b=9000, bt=cr.BF16), dict(w=8192 - 126, wt=cr.BF16), dict(w=9600)])
def test_group_norm_over_weight_or_bias(kw):
    assert group_norm._apply(batch=2, positions=3, **kw) == cr.ERR_UNSUPPORTED


@cpu_only
def test_group_norm_beside_weight_and_bias():
    # (made-up addresses: a call that passes would run)
    assert group_norm._apply(batch=2, positions=0, w=8192) == cr.OK


@pytest.mark.gpu
@pytest.mark.parametrize("positions", [4, 9000])
def test_group_norm_outputs(positions):
    c = 64
    space = torch.randn(2 * positions * c + 2 * c, device="cuda")
    out = space[c:c + 2 * positions * c].view(2, positions, c)
    x = torch.randn(2, positions, c, device="cuda")
    before, behind = space[:c], space[-c:]
    for weight, bias in ((space[1:c + 1], None), (None, space[-c - 1:-1]), (out[1, 2], behind), (before, out[0, 0])):
        with pytest.raises(ValueError, match="weight or bias"):
            cr.group_norm(x, 4, weight, bias, out=out)
    want = cr.group_norm(x, 4, before, behind)
    assert torch.equal(cr.group_norm(x, 4, before, behind, out=out), want)
