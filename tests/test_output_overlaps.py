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


# Y: [4, 64] from 2^20 on, rows 80 apart, bfloat16 or float32; the gate's codes 64 x 128 from 2^16 on, ...
PAIR = dict(gate=dict(q=1 << 16, scale=1 << 17, bias=1 << 18), up=dict(q=(1 << 16) + 8192, scale=(1 << 17) + 16),
            y=1 << 20, ldy=80)
Y_BYTES = (3 * 80 + 64) * 2


def _pair(call=gated._gated, **kw):
    kw = {**PAIR, **kw}
    for which in ("gate", "up"):
        kw[which] = {**PAIR[which], **kw.get(which, {})}
    return call(m=4, **kw)


@cpu_only
@pytest.mark.parametrize("call", [gated._gated, gated._rows])
@pytest.mark.parametrize("kw", [
    dict(gate=dict(q=1 << 20)), dict(up=dict(q=(1 << 20) + Y_BYTES - 16 - Y_BYTES % 16)), dict(up=dict(q=(1 << 20) - 8176)),
    dict(gate=dict(scale=1 << 20)), dict(up=dict(scale=(1 << 20) + Y_BYTES - 1)), dict(up=dict(bias=(1 << 20) - 252)),
    dict(y_dtype=cr.F32, gate=dict(bias=(1 << 20) + 2 * Y_BYTES - 4)),
    dict(kept_gate=1 << 22, kept_up=1 << 18), dict(kept_gate=(1 << 16) + 8192, kept_up=1 << 22)])
def test_gated_over_its_weights(call, kw):
    assert _pair(call, **kw) == cr.ERR_UNSUPPORTED


@cpu_only
def test_gated_over_a_packed_x():
    for y in (4096, 4096 + 508, 8192):
        x = gated._packed(m=4, q=4096, scale=8192)
        assert cr.lib().convrot_fp8_gated(x, gated._pair(**{**PAIR, "y": y}), None) == cr.ERR_UNSUPPORTED


@pytest.mark.gpu
@pytest.mark.parametrize("m", [3, 100])
def test_gated_outputs(m):
    n = k = 256
    space = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    out = space[4096:4096 + 2 * m * n].view(BF16).view(m, n)
    w = cr.fp8_quantize_weights(torch.randn(n, k, device="cuda"))
    x = torch.randn(m, k, device="cuda")
    over = cr.Fp8Weights(space[:n * k].view(torch.float8_e4m3fn).view(n, k), w.scale)
    for gate, up in ((over, w), (w, over), (w, cr.Fp8Weights(w.q, w.scale, space[4096:4096 + 4 * n].view(F32)))):
        with pytest.raises(cr.ConvrotError):
            cr.fp8_gated(x, gate, up, out=out)
    packed = cr.fp8_pack_activations(x)
    space[4096:4096 + m * k] = packed.q.view(torch.uint8).view(-1)
    with pytest.raises(cr.ConvrotError):
        cr.fp8_gated(cr.Fp8Activation(space[4096:4096 + m * k].view(torch.float8_e4m3fn).view(m, k), packed.scale),
                     w, w, out=out)
    assert torch.equal(cr.fp8_gated(x, w, w, out=out), cr.fp8_gated(x, w, w, out_dtype=BF16))


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
