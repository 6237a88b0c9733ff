"""Group norm against its definition in 64 bits: group sizes on both sides of what a workgroup holds,
odd channels, types, strides, a large common part, captured calls and other streams."""

import math

import pytest
import torch

import hadamard_rotated_int8_amd as cr

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _reference(x, groups, weight, bias, eps, silu, y_dtype):
    """(y, tol) in float64.

    The mean comes out within 256 2^-24 of the deviation and of the distance of the group's first value
    (sums of at most 64 values a thread, 6 + 16 more in a workgroup; in runs of positions, a union for
    every 8 rows of a thread, all relative to that value), the variance to twice that of its size.
    SiLU's slope is at most 1.1 and its own error 2^-21 of its value.
    """
    b, c = x.shape[0], x.shape[-1]
    v = x.double().reshape(b, -1, groups, c // groups)
    mean = v.mean(dim=(1, 3), keepdim=True)
    dev = ((v - mean) ** 2).mean(dim=(1, 3), keepdim=True)
    first = (v[:, :1, :, :1] - mean).abs() / (dev + eps).sqrt()
    n = (v - mean) / (dev + eps).sqrt()
    tol = 256 * 2.0 ** -24 * (1 + n.abs()) * (1 + first)
    n, tol = (t.reshape(b, -1, c) for t in (n, tol))
    if weight is not None:
        n, tol = n * weight.double(), tol * weight.double().abs()
    if bias is not None:
        n, tol = n + bias.double(), tol + 2.0 ** -23 * (bias.double().abs() + n.abs())
    if silu:
        n = n * torch.sigmoid(n)
        tol = 1.1 * tol + 2.0 ** -21 * n.abs()
    tol = tol + n.abs() * torch.finfo(y_dtype).eps / 2 + 1e-30
    return n.reshape(x.shape), tol.reshape(x.shape)


def _check(x, groups, weight=None, bias=None, eps=1e-6, silu=False, out_dtype=None, **kw):
    y = cr.group_norm(x, groups, weight, bias, eps=eps, silu=silu, out_dtype=out_dtype, **kw)
    ref, tol = _reference(x, groups, weight, bias, eps, silu, y.dtype)
    assert y.shape == x.shape and y.dtype == (out_dtype or x.dtype)
    off = (y.double() - ref).abs()
    assert not y.isnan().any() and (off <= tol).all(), ((off - tol).max().item(), off.max().item())
    return y


def _x(*shape, dtype=torch.float32, seed=0, mean=0.25):
    g = torch.Generator(device=DEV).manual_seed(seed)
    channels = torch.exp(torch.randn(shape[-1], generator=g, device=DEV))
    return (torch.randn(*shape, generator=g, device=DEV) * channels + mean).to(dtype)


def _affine(c, dtype, seed=1):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return ((1 + 0.1 * torch.randn(c, generator=g, device=DEV)).to(dtype),
            (0.1 * torch.randn(c, generator=g, device=DEV)).to(dtype))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("batch, positions, c, groups", [
    (1, 1, 1, 1), (1, 1, 8, 2), (2, 3, 7, 7), (1, 2, 2560, 32), (3, 64, 1280, 32), (2, 63, 320, 32),
    (2, 100, 96, 32), (2, 101, 63, 3), (1, 1000, 33, 1),
    # around what a workgroup holds: 65536 values, 32768 with odd channels
    (1, 8192, 8, 1), (1, 8193, 8, 1), (2, 4096, 64, 4), (2, 4097, 64, 4), (1, 4096, 16, 2),
    (1, 16384, 2, 1), (1, 16385, 2, 1), (1, 32768, 3, 3), (1, 32769, 3, 3), (1, 1561, 63, 3), (1, 1562, 63, 3),
    # many positions, channels that fill no thread, more than one step of rows
    (1, 70001, 24, 4), (2, 40000, 129, 3), (1, 5000, 1027, 13), (1, 3000, 4096, 32), (3, 9001, 320, 10),
    (1, 300, 4095, 1), (5, 33333, 10, 5), (1, 50001, 24, 1), (2, 50000, 14, 2)])
def test_sizes(batch, positions, c, groups, silu, dtype):
    x = _x(batch, positions, c, dtype=dtype, seed=positions + c)
    weight, bias = _affine(c, dtype)
    _check(x, groups, weight, bias, silu=silu)


@pytest.mark.parametrize("x_dtype, y_dtype", [(torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("positions", [50, 30000])
def test_types(x_dtype, y_dtype, positions):
    x = _x(2, positions, 96, dtype=x_dtype)
    weight, bias = _affine(96, torch.bfloat16)
    _check(x, 8, weight, None, out_dtype=y_dtype)
    _check(x, 8, None, bias.float(), out_dtype=y_dtype, silu=True)
    _check(x, 8, out_dtype=y_dtype, eps=0.5)


@pytest.mark.parametrize("positions", [200, 40000])
@pytest.mark.parametrize("lift", [1e3, 1e5])
def test_a_common_part_costs_no_digits(positions, lift):
    x = _x(2, positions, 64, mean=0.0) + lift  # (its own rounding is part of the input)
    _check(x, 8)


@pytest.mark.parametrize("positions", [300, 40000])
def test_a_first_value_far_from_the_others(positions):
    x = _x(1, positions, 32)
    x[0, 0] = 500.0
    _check(x, 4)


@pytest.mark.parametrize("positions", [64, 40000])
def test_nan_and_constant_groups(positions):
    x = _x(2, positions, 32)
    x[0, positions // 2, 5] = math.nan
    x[1, :, 8:16] = 3.5
    x[1, positions - 1, 20] = math.inf
    y = cr.group_norm(x, 4)
    assert y[0, :, :8].isnan().all() and not y[0, :, 8:].isnan().any()
    assert (y[1, :, 8:16] == 0).all()
    assert y[1, :, 16:24].isnan().all() and not y[1, :, 24:].isnan().any() and not y[1, :, :8].isnan().any()


@pytest.mark.parametrize("h, w", [(5, 9), (200, 201)])
def test_layouts_and_outputs(h, w):
    x = _x(2, 48, h, w).to(memory_format=torch.channels_last)
    nhwc = x.permute(0, 2, 3, 1)
    weight, bias = _affine(48, torch.float32)
    ref = _check(nhwc.contiguous(), 6, weight, bias)
    assert torch.equal(_check(nhwc, 6, weight, bias), ref)
    wide = torch.full((2, h * w, 50), 7.0, device=DEV)
    out = wide[:, :, 1:49]
    assert cr.group_norm(nhwc.reshape(2, h * w, 48), 6, weight, bias, out=out) is out
    assert torch.equal(out, ref.reshape(out.shape))
    out.fill_(7.0)
    assert (wide == 7.0).all()
    part = torch.randn(2, h * w, 60, device=DEV)[:, :, 5:53]
    _check(part, 6, weight, bias)
    copy = nhwc.contiguous()
    assert cr.group_norm(copy, 6, weight, bias, out=copy) is copy
    assert torch.equal(copy, ref)


@pytest.mark.parametrize("positions", [64, 40000])
def test_graphs_and_streams(positions):
    x = _x(2, positions, 64, dtype=torch.bfloat16)
    weight, bias = _affine(64, torch.float32)
    want = cr.group_norm(x, 8, weight, bias, silu=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = cr.group_norm(x, 8, weight, bias, silu=True)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res = cr.group_norm(x, 8, weight, bias, silu=True)
        graphs.append((graph, res))
    for round in range(3):
        x.copy_(_x(2, positions, 64, dtype=torch.bfloat16, seed=round + 5))
        eager = cr.group_norm(x, 8, weight, bias, silu=True)
        for graph, res in graphs:
            res.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(res, eager)


def test_empty_sizes():
    assert cr.group_norm(torch.empty(0, 5, 8, device=DEV), 2).shape == (0, 5, 8)
    assert cr.group_norm(torch.empty(2, 0, 8, device=DEV), 2).shape == (2, 0, 8)


def test_refusals():
    x = _x(2, 30, 8, 6)
    for bad, kw in [((x, 4), {}), ((x, 0), {}), ((x.transpose(1, 2), 2), {}), ((x.half(), 2), {}),
                    ((x[:, :, 0, 0], 2), {}), ((x, 2), dict(out_dtype=torch.float16)),
                    ((x, 2), dict(out=x[:, :, :, :3])), ((x, 2), dict(weight=x[0, 0, 0, :3])),
                    ((x[:, :, 1:], 2), dict(out=x[:, :, :-1])), ((x, 2), dict(out=x[:1].expand_as(x)))]:
        with pytest.raises(ValueError):
            cr.group_norm(*bad, **kw)
    with pytest.raises(cr.ConvrotError):
        cr.group_norm(x, 2, eps=-1.0)
