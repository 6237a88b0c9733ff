"""Calls that the documentation of the block operators allows and that are easily missed (GPU)."""

import pytest
import torch

import hadamard_rotated_int8_amd as cr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    cr.lib()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_one_row_starts_at_a_multiple_of_16_bytes_and_that_is_all(dtype):
    """The distance to a next row that is not there says nothing."""
    k = 400
    x = torch.randn(1, k + 3, device="cuda").to(dtype)[:, :k]
    assert x.stride(0) * x.element_size() % 16
    w = cr.fp8_quantize_weights(torch.randn(70, k, device="cuda"))
    same = x.clone(memory_format=torch.contiguous_format)
    p, q = cr.fp8_pack_activations(x), cr.fp8_pack_activations(same)
    assert torch.equal(p.q.view(torch.uint8), q.q.view(torch.uint8))
    assert torch.equal(p.scale.view(torch.uint8), q.scale.view(torch.uint8))
    assert torch.equal(cr.fp8_linear(x, w), cr.fp8_linear(same, w))
    with pytest.raises(cr.ConvrotError):  # two rows do need it
        cr.fp8_pack_activations(torch.randn(2, k + 3, device="cuda").to(dtype)[:, :k])
