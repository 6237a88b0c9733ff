"""Operators without a gradient say so where autograd comes back to them."""

import pytest
import torch

import hadamard_rotated_int8_amd as cr
from hadamard_rotated_int8_amd import block as impl

BF16 = torch.bfloat16


def _twice(x):
    return 2 * x


def test_going_back_raises():
    x = torch.ones(3, requires_grad=True)
    y = impl._NoGradient.apply(_twice, (x,), "use g", x, None)
    assert y.requires_grad and torch.equal(y.detach(), torch.full((3,), 2.0))
    with pytest.raises(NotImplementedError, match="_twice records no gradient: use g"):
        (y.sum() + x.sum()).backward()


def test_outputs_are_refused():
    x = torch.ones(3, requires_grad=True)
    with pytest.raises(ValueError, match="out cannot be given"):
        impl._no_gradient(_twice, (x,), "use g", torch.empty(3), x)


def _calls():
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(2, n, 2, 64, generator=g, device="cuda").to(BF16) for n in (5, 40, 40))
    x, w = torch.randn(2, 9, 32, generator=g, device="cuda"), torch.randn(32, generator=g, device="cuda")
    rows, bias = torch.randn(4, 64, generator=g, device="cuda"), torch.randn(48, generator=g, device="cuda")
    code = cr.fp8_quantize_weights(torch.randn(48, 64, generator=g, device="cuda"))

    def gated(a, b, keep):
        return cr.fp8_gated(a, cr.Fp8Weights(code.q, code.scale, b), code, keep=keep)

    return {
        "attention": ([q, k, v], lambda a, b, c: cr.attention(a, b, c)),
        "group_norm": ([x, w, w], lambda a, b, c: cr.group_norm(a, 4, b, c, silu=True)),
        "fp8_gated": ([rows, bias], lambda a, b: gated(a, b, False)),
        "fp8_gated keep": ([rows, bias], lambda a, b: gated(a, b, True)[0]),
    }


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["attention", "group_norm", "fp8_gated", "fp8_gated keep"])
def test_no_gradient_vanishes(name):
    inputs, call = _calls()[name]
    want = call(*inputs)
    assert not want.requires_grad
    for i in range(len(inputs)):
        leaves = [t.clone().requires_grad_(j == i) for j, t in enumerate(inputs)]
        with torch.no_grad():
            assert not call(*leaves).requires_grad
        y = call(*leaves)
        assert y.requires_grad and torch.equal(y.detach(), want)
        with pytest.raises(NotImplementedError, match=name.split()[0]):
            y.float().sum().backward()


@pytest.mark.gpu
def test_kept_projections_and_outputs():
    n, k = 48, 64
    w = cr.fp8_quantize_weights(torch.randn(n, k, device="cuda"))
    x = torch.randn(4, k, device="cuda", requires_grad=True)
    y, kept = cr.fp8_gated(x, w, w, keep=True)
    assert y.requires_grad and not any(t.requires_grad for t in kept)
    dx, _ = cr.fp8_gated_backward(torch.ones(4, n, device="cuda"), kept, cr.fp8_transpose_weights([w, w]))
    assert dx.shape == x.shape
    with pytest.raises(ValueError, match="out cannot be given"):
        cr.fp8_gated(x, w, w, out=torch.empty(4, n, device="cuda"))
    with torch.no_grad():
        assert torch.equal(cr.fp8_gated(x, w, w, out=torch.empty(4, n, device="cuda")), y)


class _Gated(torch.autograd.Function):  # as a caller writes it
    @staticmethod
    def forward(ctx, x, gate, up, back):
        y, kept = cr.fp8_gated(x, gate, up, keep=True)
        ctx.kept, ctx.back = kept, back
        return y

    @staticmethod
    def backward(ctx, dy):
        return cr.fp8_gated_backward(dy.contiguous(), ctx.kept, ctx.back)[0].to(dy.dtype), None, None, None


@pytest.mark.gpu
def test_a_callers_own_function_goes_back():
    n, k = 256, 128
    gate, up = (cr.fp8_quantize_weights(torch.randn(n, k, device="cuda")) for _ in range(2))
    back = cr.fp8_transpose_weights([gate, up])
    x = torch.randn(8, k, device="cuda", requires_grad=True)
    dy = torch.randn(8, n, device="cuda")
    _Gated.apply(x, gate, up, back).backward(dy)
    kept = cr.fp8_gated(x.detach(), gate, up, keep=True)[1]
    assert torch.equal(x.grad, cr.fp8_gated_backward(dy, kept, back)[0].float())


@pytest.mark.gpu
def test_no_second_gradient_vanishes():
    n, k = 256, 128
    gate, up = (cr.fp8_quantize_weights(torch.randn(n, k, device="cuda")) for _ in range(2))
    back = cr.fp8_transpose_weights([gate, up])
    kept = cr.fp8_gated(torch.randn(8, k, device="cuda"), gate, up, keep=True)[1]
    dy = torch.randn(8, n, device="cuda")
    want, (dg, du) = cr.fp8_gated_backward(dy, kept, back)
    dx, grads = cr.fp8_gated_backward(dy.clone().requires_grad_(), kept, back)
    assert dx.requires_grad and torch.equal(dx.detach(), want)
    assert torch.equal(grads[0].detach(), dg) and torch.equal(grads[1].detach(), du)
    for t in (dx, *grads):
        with pytest.raises(NotImplementedError, match="fp8_gated_backward"):
            t.float().sum().backward(retain_graph=True)
