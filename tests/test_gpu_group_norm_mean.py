"""Group norm of groups whose first values are far from the others: the mean comes off without their
rounding (GPU)."""

import pytest
import torch

import hadamard_rotated_int8_amd as cr

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _check(x, groups, y):
    """y against its definition in 64 bits, no value's error depending on another value.

    A difference from the mean is off by 2^-23 of itself and by the mean's own error, which is that of the
    threads' means of at most 8 blocks of 4 rows: each takes 8 roundings of at most the deviation, whatever
    a single value is (what a far value costs its own thread is shared out over the group).  The variance is
    off by 2^-19 of itself at most (32 roundings), its root by half of that; scale and product take 3 more.
    """
    b, c = x.shape[0], x.shape[-1]
    v = x.double().reshape(b, -1, groups, c // groups)
    mean = v.mean(dim=(1, 3), keepdim=True)
    dev = ((v - mean) ** 2).mean(dim=(1, 3), keepdim=True)
    n = ((v - mean) / (dev + 1e-6).sqrt()).reshape(x.shape)
    off = (y.double() - n).abs()
    tol = 2.0 ** -24 * (64 + 24 * n.abs())
    assert (off <= tol).all(), ((off - tol).max().item(), off.max().item())


def _x(positions, c, lift=0.0):
    g = torch.Generator(device=DEV).manual_seed(positions + c)
    return torch.randn(1, positions, c, generator=g, device=DEV) + lift


@pytest.mark.parametrize("positions, c, groups", [
    (1000, 32, 4), (40000, 32, 4), (131072, 32, 1), (16400, 320, 32), (50001, 24, 1), (30000, 21, 3)])
@pytest.mark.parametrize("far", [2e3, -3e4, 1e6])
def test_a_first_value_far_from_the_others(positions, c, groups, far):
    x = _x(positions, c)
    x[0, 0, 0] = far
    _check(x, groups, cr.group_norm(x, groups))


@pytest.mark.parametrize("positions, c, groups", [(1000, 32, 4), (40000, 32, 4), (131072, 32, 1), (30000, 21, 3)])
@pytest.mark.parametrize("at", [0, 1, 517, -1])
def test_a_position_far_from_the_others(positions, c, groups, at):
    x = _x(positions, c)
    x[0, at] *= 5e3
    _check(x, groups, cr.group_norm(x, groups))


@pytest.mark.parametrize("lift", [0.0, 300.0, -7e4])
def test_far_values_beside_a_common_part(lift):
    x = _x(60000, 64, lift)
    x[0, 0] = 5e5
    x[0, 3, ::7] = -2e5
    x[0, 40000, 5] = 1e6
    _check(x, 8, cr.group_norm(x, 8))
