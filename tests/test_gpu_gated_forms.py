"""The gated pair in the shapes of tiles that test_gpu_gated.py's sizes do not reach, edges of the large tiles
with float32 scales among them; and which kernel takes which sizes (GPU)."""

import pytest
import torch

import hadamard_rotated_int8_amd as cr
from kernel_names import launched
from test_gpu_gated import BF16, DTYPES, E8M0, F32, SCALES, _check, _weights, _x

pytestmark = pytest.mark.gpu


def _run(m, k, n, scale, dtype, act, keep):
    gate, up = _weights(n, k, scale, n + k), _weights(n, k, scale, n + k + 1, bias=n % 2 == 0)
    x = _x(m, k, BF16, m + k)
    got = cr.fp8_gated(x, gate, up, act=act, out_dtype=dtype, keep=keep)
    y, kept = got if keep else (got, None)
    _check(x, gate, up, act, dtype, y, kept)
    return launched(lambda: cr.fp8_gated(x, gate, up, act=act, out_dtype=dtype, keep=keep))[-1]


def _gemm(shape, scale, dtype):
    flags = ", ".join(str(f).lower() for f in (scale == F32, dtype == F32, True))
    return f"fp8_gemm_kernel<{shape}, {flags}>"


@SCALES
@DTYPES
@pytest.mark.parametrize("act, keep", [("silu", True), ("gelu", False)])
@pytest.mark.parametrize("m, k, n, shape", [
    (64, 400, 8200, "1, 1, 2, 2, 1, 3"), (33, 640, 13001, "1, 1, 2, 2, 1, 3"), (50, 5120, 8256, "1, 1, 2, 2, 1, 3"),
    (200, 400, 4090, "2, 1, 2, 2, 2, 3"), (129, 1040, 3999, "2, 1, 2, 2, 2, 3")])
def test_shapes_of_tiles(m, k, n, shape, scale, dtype, act, keep):
    assert _run(m, k, n, scale, dtype, act, keep) == _gemm(shape, scale, dtype)


@pytest.mark.parametrize("act, keep", [("silu", True), ("gelu", True), ("silu", False)])
@pytest.mark.parametrize("m, k, n", [(1000, 384, 4000), (900, 656, 3990), (1023, 400, 4033), (1900, 400, 8100)])
def test_edges_of_large_tiles_with_float32_scales(m, k, n, act, keep):
    assert m % 256 and n % 64
    assert _run(m, k, n, F32, BF16, act, keep) == f"fp8_gated_wide_kernel<true, {2 if keep else 1}>"


@pytest.mark.parametrize("act, keep", [("silu", True), ("gelu", False)])
@pytest.mark.parametrize("m, k, n", [(1100, 400, 8200), (2100, 656, 4001)])
def test_edges_of_large_tiles(m, k, n, act, keep):
    assert _run(m, k, n, E8M0, BF16, act, keep) == f"fp8_gated_wide_kernel<false, {2 if keep else 1}>"


@SCALES
def test_outputs_of_wider_rows(scale):
    # rows that allow no vector stores, and rows that do, in each shape of tiles above
    for m, k, n in ((64, 400, 8200), (200, 400, 4090), (1000, 384, 4000)):
        gate, up = _weights(n, k, scale, 1), _weights(n, k, scale, 2)
        p = cr.fp8_pack_activations(_x(m, k, F32, 3))
        want = cr.fp8_gated(p, gate, up, out_dtype=BF16)
        for pad in (3, 8):
            wide = torch.full((m, n + 2 * pad), 7.0, dtype=BF16, device="cuda")
            assert torch.equal(cr.fp8_gated(p, gate, up, out=wide[:, pad:pad + n]), want)
            assert (wide[:, :pad] == 7).all() and (wide[:, pad + n:] == 7).all()


@SCALES
@DTYPES
@pytest.mark.parametrize("m, k, n, shapes", [
    (17, 1024, 2000, {BF16: "1, 1, 1, 1, 4, 3", F32: "1, 1, 1, 1, 8, 2"}), (64, 1024, 4000, "1, 1, 1, 2, 4, 3"),
    (64, 1024, 8000, "1, 1, 2, 2, 2, 3"), (333, 640, 4104, {BF16: "2, 1, 2, 4, 1, 4", F32: "1, 2, 4, 2, 2, 2"}),
    (600, 256, 8000, "2, 2, 2, 2, 1, 2")])
def test_which_kernel(m, k, n, shapes, scale, dtype):
    if torch.cuda.get_device_properties(0).multi_processor_count != 256:
        pytest.skip("the rule goes by the compute units")
    gate, up = _weights(n, k, scale, 1), _weights(n, k, scale, 2)
    p = cr.fp8_pack_activations(_x(m, k, F32, 3))
    names = launched(lambda: cr.fp8_gated(p, gate, up, out_dtype=dtype))
    assert names == [_gemm(shapes if isinstance(shapes, str) else shapes[dtype], scale, dtype)]
