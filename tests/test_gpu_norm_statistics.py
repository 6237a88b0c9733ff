"""The statistics of the norms around a block where they are most easily wrong: rows with a large
common part, rows whose size is that of eps, rows of one value (GPU).

Tolerances, with u = 2^-24 and sums that go through at most 64 roundings relative to their magnitudes
(test_gpu_block_norm.py).  A layer norm's first mean is off by D <= 64 u mean|v|.  The centred values
d = v - mean are rounded by u |d|; their own mean, which takes that D off again, by 66 u mean|d|; and
their difference by u once more, where |d| <= |c| + D (c the exact centred values).  So a value is off
by at most 70 u (1 + D / rms(c)) of rms(c), and by 2 u of itself.  The mean square, sum d^2 / k less
that mean's square, is off by 66 u (1 + D / rms(c))^2 of itself, its root by half, the division, root
and product by 4 u.  With eps the root is of a larger number, which makes all of it smaller:
    |n^ - n| <= 128 u (1 + D / rms(c))^2 (1 + |n|) in units of n's scale.
"""

import pytest
import torch

import block_reference as ref
import hadamard_rotated_int8_amd as cr

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    cr.lib()
    yield
    torch.cuda.synchronize()


def _tolerance(v, n, kind, eps):
    """The module's bound for n, the norm of v (float64 rows)."""
    c = v - v.mean(1, keepdim=True) if kind == "layer" else v
    rms = ((c * c).mean(1, keepdim=True) + eps).sqrt()
    d = 64 * U * v.abs().mean(1, keepdim=True) / rms if kind == "layer" else 0
    return 128 * U * (1 + d) ** 2 * (1 + n.abs())


@pytest.mark.parametrize("k", [64, 500, 1031, 2048, 5120, 9001, 32768])
@pytest.mark.parametrize("offset", [0.0, 1.0, -300.0, 4096.0, -1e5])
def test_a_common_part_costs_no_digits(k, offset):
    print(f"[gpu] block_norm offset {offset} {k}", flush=True)
    g = torch.Generator().manual_seed(k)
    x = (offset + torch.randn(7, k, generator=g)).float()
    for x in (x, x.to(torch.bfloat16)):
        if ((x.double() - x.double().mean(1, keepdim=True)) ** 2).mean() < 0.01:
            continue  # (in bfloat16 nothing but the offset is left)
        want = ref.norm(x, "layer", 1e-6)
        y = cr.block_norm(x.cuda(), cr.Norm("layer", 1e-6), out_dtype=torch.float32).cpu().double()
        assert ((y - want).abs() <= _tolerance(x.double(), want, "layer", 1e-6)).all()
        # the second norm of an update, on h as it is before it is rounded
        zero = torch.zeros_like(x)
        _, y = cr.block_update(x.cuda(), zero.cuda(), norm=cr.Norm("layer", 1e-6), out_dtype=torch.float32)
        assert ((y.cpu().double() - want).abs() <= _tolerance(x.double(), want, "layer", 1e-6)).all()


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("k", [8, 333, 4096])
def test_rows_of_the_size_of_eps(k, kind):
    """eps decides the result: another one, the other norm's or none would be off by far more."""
    print(f"[gpu] block_norm eps {k} {kind}", flush=True)
    g = torch.Generator().manual_seed(k)
    for eps in (1e-2, 1e-5, 1e-12):
        x = (torch.randn(5, k, generator=g) * eps ** 0.5).float()
        want = ref.norm(x, kind, float(torch.tensor(eps)))
        y = cr.block_norm(x.cuda(), cr.Norm(kind, eps)).cpu().double()
        assert ((y - want).abs() <= _tolerance(x.double(), want, kind, eps)).all()
        assert ((want - ref.norm(x, kind, eps / 4)).abs().amax(1) > 0.1 * want.abs().amax(1)).all()


@pytest.mark.parametrize("post,pre", [("rms", "layer"), ("layer", "rms")])
def test_each_norm_has_its_own_eps(post, pre):
    """h = x + post(branch) with rows that make post's eps count, y = pre(h) with one that makes pre's
    count.  h is float32 and exact to 128 u (1 + |n|) of post's n and a rounding; y is then pre of the
    h that came out, which differs from the h it was computed from by nothing (float32)."""
    k = 1000
    g = torch.Generator().manual_seed(1)
    a, b = 1e-2, 3.0
    x = torch.randn(6, k, generator=g).float()
    branch = (torch.randn(6, k, generator=g) * 0.1).float()
    h, y = cr.block_update(x.cuda(), branch.cuda(), post=cr.Norm(post, a), norm=cr.Norm(pre, b))
    h, y = h.cpu().double(), y.cpu().double()
    a, b = float(torch.tensor(a)), float(torch.tensor(b))
    n = ref.norm(branch, post, a)
    assert ((h - (x.double() + n)).abs() <= _tolerance(branch.double(), n, post, a) + U * (x + n).abs()).all()
    want = ref.norm(h, pre, b)
    assert ((y - want).abs() <= _tolerance(h, want, pre, b)).all()
    assert ((want - ref.norm(h, pre, a)).abs().amax(1) > 0.1).all()
    assert ((n - ref.norm(branch, post, b)).abs().amax(1) > 0.1).all()


@pytest.mark.parametrize("xt", [torch.float32, torch.bfloat16])
def test_a_layer_norm_of_one_value_leaves_bias_and_shift(xt):
    """(v - v) / sqrt(eps) is 0 exactly: bias * (1 + scale) + shift is left, two roundings and a fused
    or separate sum."""
    g = torch.Generator().manual_seed(2)
    x = (torch.randn(70, 1, generator=g) * 100).to(xt)
    w, b, scale, shift = (torch.randn(1, generator=g) for _ in range(4))
    y = cr.block_norm(x.cuda(), cr.Norm("layer", 1e-5, w.cuda(), b.cuda()), scale.cuda(), shift.cuda(),
                      out_dtype=torch.float32).cpu().double()
    w, b, scale, shift = (t.double() for t in (w, b, scale, shift))
    want = (b * (1 + scale) + shift).expand(70, 1)
    assert ((y - want).abs() <= 4 * U * ((b * (1 + scale)).abs() + shift.abs())).all()


def test_rows_of_equal_values():
    """A constant row is its bias: what is left of rounding is far below eps' root, whatever the value."""
    for k in (3, 100, 640, 1031, 5120):
        x = torch.tensor([[0.1], [2.5], [-333.3], [1e4]]).expand(4, k).contiguous()
        y = cr.block_norm(x.cuda(), cr.Norm("layer", 1e-6)).cpu().double()
        # a mean's rounding, 64 u |v|, less its own mean: 70 u of that, over 1e-3
        assert (y.abs() <= 70 * U * 64 * U * x.double().abs() / 1e-3 + 1e-30).all()


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("k", [5, 384, 2000])
def test_a_row_with_a_nan_is_nan_and_others_are_not(k, kind):
    """As the formula has it: the statistics of such a row are NaN.  An infinity makes the root
    infinite: 0 for the other values of an rms norm, NaN for itself and for all of a layer norm's."""
    x = torch.randn(9, k)
    x[1, 3], x[7, 0], x[4, 2] = float("nan"), float("nan"), float("inf")
    n = cr.Norm(kind, 1e-6)
    y = cr.block_norm(x.cuda(), n).cpu()
    _, after = cr.block_update(x.cuda(), torch.zeros(9, k, device="cuda"), norm=n)
    h, _ = cr.block_update(torch.zeros(9, k, device="cuda"), x.cuda(), post=n)
    want = ref.norm(x, kind, 1e-6)
    assert torch.isnan(want[[1, 7]]).all()
    for got in (y, after.cpu(), h.cpu()):
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got[4].nan_to_num(1.0), want[4].float().nan_to_num(1.0))
        rest = [0, 2, 3, 5, 6, 8]
        assert ((got[rest] - want[rest]).abs() <= _tolerance(x[rest].double(), want[rest], kind, 1e-6)).all()


def test_signs_of_zero_and_rows_without_eps():
    x = torch.zeros(3, 16)
    x[0, 0], x[0, 1] = -0.0, 2.0
    x[1] = 1e-30  # squares below float32: the root is of zero
    y = cr.block_norm(x.cuda(), cr.Norm("rms", 0.0)).cpu()
    assert torch.signbit(y[0, 0]) and not torch.signbit(y[0, 2]) and y[0, 1] == 4.0
    assert torch.isinf(y[1]).all() and torch.isnan(y[2]).all()
