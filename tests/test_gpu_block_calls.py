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


@pytest.mark.parametrize("m", [1, 9, 40])
def test_a_linear_s_output_may_lie_over_its_input(m):
    """The whole of X is read before any of Y is written, however few rows it has."""
    k = 2048
    g = torch.Generator().manual_seed(m)
    ws = [cr.fp8_quantize_weights((torch.randn(n, k, generator=g) * 0.02).cuda()) for n in (k, 900)]
    x = torch.randn(m, k, generator=g).cuda()
    p = cr.fp8_pack_activations(x)
    for _ in range(3):
        y = x.clone()
        assert cr.fp8_linear(y, ws[0], out=y) is y
        assert torch.equal(y, cr.fp8_linear(p, ws[0]))
        buffer = torch.full((m, k + 1000), 2.0, device="cuda")
        a, b = buffer[:, :k], buffer[:, k:k + 900]  # one over X, one beside it
        a.copy_(x)
        cr.fp8_linear_grouped(a, ws, (a, b))
        for got, want in zip((a, b), cr.fp8_linear_grouped(p, ws)):
            assert torch.equal(got, want)
        assert (buffer[:, k + 900:] == 2).all()
