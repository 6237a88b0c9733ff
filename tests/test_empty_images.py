"""Group norm of images without a position, whatever their strides say."""

import pytest
import torch

import hadamard_rotated_int8_amd as cr
from hadamard_rotated_int8_amd.block import _positions

SHAPES = [(2, 0, 8), (2, 3, 0, 8), (2, 0, 3, 8), (2, 4, 0, 5, 8), (0, 3, 5, 8), (1, 0, 0, 8)]


@pytest.mark.parametrize("shape", SHAPES)
def test_positions(shape):
    images, positions, stride = _positions(torch.empty(shape), "x")
    assert images == shape[0] and stride == 8
    assert positions == torch.Size(shape[1:-1]).numel()


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES)
def test_group_norm(shape):
    x = torch.empty(shape, device="cuda")
    assert cr.group_norm(x, 2).shape == shape
    assert cr.group_norm(x, 2, out=x) is x
    wide = torch.empty(*shape[:-1], 16, device="cuda")
    assert cr.group_norm(wide[..., 4:12], 2).shape == shape
