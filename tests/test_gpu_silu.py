"""SiLU behind group norm and in the gated pair over the whole range of its values, against 64 bits (GPU)."""

import pytest
import torch

import hadamard_rotated_int8_amd as cr

pytestmark = pytest.mark.gpu

# To -87: exp(87) is the last power whose reciprocal is a normal number.
POINTS = torch.cat([torch.linspace(-87, 20, 3000), torch.linspace(-1, 1, 900), -torch.logspace(-30, 1.9, 150),
                    torch.tensor([-128.0, -1e3, -3e38, 88.0, 200.0, 3e38])])


def _check(y, x):
    """x sigmoid(x) within 2^-21 of itself: the exponential and the reciprocal are off by a unit in the last
    place (2^-23), the exponent's correction, two products and a sum by 2^-24 each."""
    x = x.double()
    want = x * torch.sigmoid(x)
    off = (y.double() - want).abs()
    tol = 2.0 ** -21 * want.abs() + 1e-37
    assert not y.isnan().any() and (off <= tol).all(), (off / want.abs()).max().log2()


def test_behind_group_norm():
    # a weight of zero leaves the bias
    c = POINTS.numel()
    bias = POINTS.cuda()
    for positions in (2, 300):  # a group in one workgroup, or in runs
        x = torch.randn(1, positions, c, device="cuda")
        _check(cr.group_norm(x, 1, torch.zeros_like(bias), bias, silu=True)[0], bias.expand(positions, c))


@pytest.mark.parametrize("scale", [torch.float8_e8m0fnu, torch.float32])
@pytest.mark.parametrize("m", [1, 100])
def test_in_the_gated_pair(m, scale):
    # weights of zero leave the biases, POINTS and ones
    n, k = POINTS.numel(), 128
    w = cr.fp8_quantize_weights(torch.zeros(n, k, device="cuda"))
    bias = POINTS.cuda()
    gate = cr.Fp8Weights(w.q, w.scale.to(scale), bias)
    up = cr.Fp8Weights(w.q, w.scale.to(scale), torch.ones_like(bias))
    y = cr.fp8_gated(torch.randn(m, k, device="cuda"), gate, up)
    _check(y, bias.expand(m, n))


@pytest.mark.parametrize("m", [1, 100])
def test_infinite_gates(m):
    w = cr.fp8_quantize_weights(torch.zeros(16, 128, device="cuda"))
    bias = torch.full((16,), float("inf"), device="cuda")
    up = cr.Fp8Weights(w.q, w.scale, torch.full((16,), 3.0, device="cuda"))
    for dtype in (torch.float32, torch.bfloat16):
        y = cr.fp8_gated(torch.randn(m, 128, device="cuda"), cr.Fp8Weights(w.q, w.scale, bias), up, out_dtype=dtype)
        assert (y == float("inf")).all()


def test_a_nan_stays_one():
    bias = torch.tensor([float("nan"), 1.0, -2.0], device="cuda")
    y = cr.group_norm(torch.randn(1, 5, 3, device="cuda"), 1, torch.zeros_like(bias), bias, silu=True)
    assert y[..., 0].isnan().all() and not y[..., 1:].isnan().any()
