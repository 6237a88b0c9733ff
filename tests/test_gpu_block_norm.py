"""The norms around a block with its gate and residual, against a plain 64-bit reference (GPU).

Tolerances.  With u = 2^-24 (half a float32 step), a row of k values and T
threads, a sum goes through at most k / T + 16 + 8 additions in a row, of
which each is off by u relative to the sum of magnitudes; T >= k / 32, so at
most 56, taken as 64 u.
* mean: 64 u mean|v|; a centred value is off by that and by u |v|, in all
  66 u (|v| + mean|v|) =: d.
* mean square of the centred values c: relative 64 u from the sum, 2 u from
  square and scale, and twice the centring's relative error in the 2-norm,
  so the reciprocal root is off by half: 33 u + 64 u A + 4 u with
  A = (rms(v) + mean|v|) / rms(c): in all r = (40 + 70 A) u.
* the result n = c / rms * weight + bias is off by (d / rms) |weight| plus
  (r + 4 u) |n'| plus u |n|, n' the value before the bias.
Modulation adds 2 u per factor and addend; an output's type adds half a step.
The branch's norm error goes through gate, and all of h's through the pre
norm, whose slope is at most 2 / rms(h) |weight| per value (the value itself
and the mean's and root's share in the 2-norm).  Rather than carrying that
algebra element by element, the tests bound the error of each row in the
2-norm with one constant: 128 u (1 + A) per norm, times 2 where a second norm
reads the first one's result, plus 8 u, plus half a step of the output's
type.  A wrong element, weight or row is off by far more than that.
"""

import pytest
import torch

import block_reference as ref
import hadamard_rotated_int8_amd as cr

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    cr.lib()
    yield
    torch.cuda.synchronize()


def _spread(v, kind):
    """A of the module's comment, for each row."""
    v = v.double()
    c = v - v.mean(1, keepdim=True) if kind == "layer" else v
    rms = (c * c).mean(1).sqrt()
    return ((v * v).mean(1).sqrt() + v.abs().mean(1)) / rms.clamp_min(1e-300)


def _check(got, want, dtype, rel):
    """Rows of got within rel and half a step of the type of want, in the 2-norm, and each element
    within the same of the row's size or its own."""
    got, want = got.cpu().double(), want.double()
    assert got.shape == want.shape
    assert bool(torch.isfinite(got).all())
    d = (got - want).abs()
    size = want.norm(dim=1)
    step = HALF_STEP[dtype]
    assert bool((d.norm(dim=1) <= (rel + step) * size + 1e-30).all())
    # one value's error: its own rounding, and at most the row's whole relative error
    assert bool((d <= step * want.abs() + rel.unsqueeze(1) * size.unsqueeze(1) + 1e-30).all())


def _rows(m, k, dtype, seed, mean=0.3):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(m, k, generator=g) * torch.exp(torch.randn(k, generator=g)) + mean
    return x.to(dtype)


def _vec(g, *shape, dtype=torch.float32):
    return (torch.randn(*shape, generator=g) * 0.3).to(dtype)


KS = [1, 2, 7, 8, 63, 128, 500, 1031, 4096, 5120, 8200, 9001, 16400, 32768]


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("k", KS)
@pytest.mark.parametrize("xt,yt", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                   (torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)])
def test_block_norm(k, kind, xt, yt):
    m = 6
    print(f"[gpu] block_norm {m}x{k} {kind} {xt}->{yt}", flush=True)
    if k == 1 and kind == "layer":
        pytest.skip("a layer norm of one value is 0 / sqrt(eps): nothing to compare relatively")
    g = torch.Generator().manual_seed(k)
    x = _rows(m, k, xt, k)
    w, b = _vec(g, k) + 1, _vec(g, k, dtype=torch.bfloat16)
    scale, shift = _vec(g, 3, 2 * k)[:, :k], _vec(g, 2 * k)[k:]
    y = cr.block_norm(x.cuda(), cr.Norm(kind, 1e-5, w.cuda(), b.cuda()), scale.cuda(), shift.cuda(),
                      out_dtype=yt)
    _, want = ref.block(x, pre=(kind, 1e-5, w, b), scale=scale, shift=shift)
    # the shift and bias may cancel the rest: the error is that of the parts
    parts = ref.norm(x, kind, 1e-5, w).abs() * (1 + ref.rows_of(scale, m)).abs() + \
        (b.double() * (1 + ref.rows_of(scale, m))).abs() + ref.rows_of(shift, m).abs()
    grown = parts.norm(dim=1) / want.norm(dim=1)
    _check(y, want, yt, (128 * (1 + _spread(x, kind)) + 8) * U * grown)


@pytest.mark.parametrize("post", [None, "layer", "rms"])
@pytest.mark.parametrize("pre", [None, "layer", "rms"])
@pytest.mark.parametrize("m,k", [(1, 5120), (4, 96), (9, 1031), (6, 12288)])
@pytest.mark.parametrize("xt,bt", [(torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16),
                                   (torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32)])
def test_block_update(m, k, post, pre, xt, bt):
    print(f"[gpu] block_update {m}x{k} post={post} pre={pre} {xt} {bt}", flush=True)
    g = torch.Generator().manual_seed(m * k)
    x, branch = _rows(m, k, xt, 1), _rows(m, k, bt, 2, mean=-0.1)
    groups = 3 if m % 3 == 0 else 1
    gate, scale, shift = (_vec(g, groups, k) for _ in range(3))
    w, b = _vec(g, k) + 1, _vec(g, k)
    h, y = cr.block_update(x.cuda(), branch.cuda(), gate.cuda(), 0.5,
                           post=post and cr.Norm(post, 1e-6, w.cuda(), b.cuda()),
                           norm=pre and cr.Norm(pre, 1e-6), scale=scale.cuda() if pre else None,
                           shift=shift.cuda() if pre else None, out_dtype=torch.float32)
    want_h, want_y = ref.block(x, branch, gate, 0.5, post and (post, 1e-6, w, b),
                               pre and (pre, 1e-6), scale if pre else None, shift if pre else None)
    parts = 0.5 * x.double().abs() + ref.rows_of(gate, m).abs() * (
        branch.double().abs() if post is None else
        ref.norm(branch, post, 1e-6, w).abs() + b.double().abs())
    grown_h = parts.norm(dim=1) / want_h.norm(dim=1)
    rel_h = (128 * (1 + _spread(branch, post)) if post else 0 * grown_h) * U * grown_h + 8 * U * grown_h
    _check(h, want_h, xt, rel_h)
    assert (y is None) == (pre is None)
    if pre:
        parts = ref.norm(want_h, pre, 1e-6).abs() * (1 + ref.rows_of(scale, m)).abs() + \
            ref.rows_of(shift, m).abs()
        grown = parts.norm(dim=1) / want_y.norm(dim=1)
        a = 1 + _spread(want_h, pre)
        _check(y, want_y, torch.float32, (2 * rel_h * a * 1.3 / 0.7 + (128 * a + 8) * U) * grown * 4)


def test_large_common_offset():
    """A layer norm of rows whose values differ by 2^-12 of their common part: the statistics are
    taken of differences, so what is lost is the input's own rounding only."""
    g = torch.Generator().manual_seed(3)
    x = (4096 + torch.randn(5, 2048, generator=g)).float()
    y = cr.block_norm(x.cuda(), cr.Norm("layer", 1e-6))
    _, want = ref.block(x, pre=("layer", 1e-6))
    _check(y, want, torch.float32, 128 * (1 + _spread(x, "layer")) * U)


def test_constant_and_zero_rows():
    x = torch.zeros(3, 640)
    x[1] = 2.5
    for kind in ("layer", "rms"):
        y = cr.block_norm(x.cuda(), cr.Norm(kind, 1e-6)).cpu()
        _, want = ref.block(x, pre=(kind, 1e-6))
        assert (y[0] == 0).all()
        assert torch.allclose(y.double(), want, rtol=64 * U, atol=0)
    # no eps: a row of zeros has no direction, 0 / 0
    assert torch.isnan(cr.block_norm(x.cuda(), cr.Norm("rms", 0.0)).cpu()[0]).all()


def test_rows_that_are_not_finite_stay_alone():
    x = torch.randn(4, 384)
    x[1, 7] = float("nan")
    x[2, 9] = float("inf")
    y = cr.block_norm(x.cuda(), cr.Norm("layer")).cpu()
    _, want = ref.block(x, pre=("layer", 1e-6))
    assert torch.isnan(y[1]).all() and torch.isnan(y[2]).any()
    assert torch.isfinite(y[[0, 3]]).all()
    assert torch.allclose(y[[0, 3]].double(), want[[0, 3]], rtol=1e-4, atol=1e-4)


@pytest.mark.parametrize("k", [16, 144, 1040, 5120, 9008, 16384])
def test_packed_output_is_the_pack_of_the_float32_output(k):
    """The FP8 output is the pack of y before y is rounded to a type: the same kernel's float32 y,
    packed by the reference."""
    print(f"[gpu] block_norm pack {k}", flush=True)
    g = torch.Generator().manual_seed(k)
    x, branch = _rows(5, k, torch.bfloat16, k), _rows(5, k, torch.float32, k + 1)
    args = dict(norm=cr.Norm("layer", 1e-6), scale=_vec(g, k).cuda(), shift=_vec(g, k).cuda())
    y = cr.block_norm(x.cuda(), out_dtype=torch.float32, **args)
    p = cr.block_norm(x.cuda(), pack=True, **args)
    d, byte = ref.pack(y.cpu())
    assert torch.equal(p.scale.contiguous().view(torch.uint8).cpu().int(), byte.int())
    assert torch.equal(ref.dequantised_rows(p.q, p.scale), d)
    h, y = cr.block_update(x.cuda(), branch.cuda(), post=cr.Norm("rms"), out_dtype=torch.float32, **args)
    h2, p = cr.block_update(x.cuda(), branch.cuda(), post=cr.Norm("rms"), pack=True, **args)
    d, byte = ref.pack(y.cpu())
    assert torch.equal(h, h2)
    assert torch.equal(p.scale.contiguous().view(torch.uint8).cpu().int(), byte.int())
    assert torch.equal(ref.dequantised_rows(p.q, p.scale), d)


def test_strides_alignment_and_in_place():
    """Rows at any element offset and stride, outputs in place or between other columns."""
    for k in (333, 1024):
        g = torch.Generator().manual_seed(k)
        wide = _rows(12, 3 * k + 5, torch.bfloat16, k).cuda()
        x, branch = wide[::2, 1:1 + k], _rows(6, 2 * k + 1, torch.float32, 7).cuda()[:, k + 1:]
        gate = _vec(g, 6, 3 * k)[:, k:2 * k]  # one row for each token
        scale = _vec(g, 2, k, dtype=torch.bfloat16)
        want_h, want_y = cr.block_update(x.contiguous(), branch.contiguous(), gate.contiguous().cuda(),
                                         norm=cr.Norm("rms"), scale=scale.cuda())
        before = wide.clone()
        y = torch.full((6, k + 7), 3.0, dtype=torch.bfloat16, device="cuda")
        h, got = cr.block_update(x, branch, gate.cuda(), norm=cr.Norm("rms"), scale=scale.cuda(),
                                 out_h=x, out=y[:, 3:3 + k])
        assert h is x and torch.equal(x, want_h) and torch.equal(got, want_y)
        before[::2, 1:1 + k] = want_h
        assert torch.equal(wide, before)  # nothing beside the rows
        assert (y[:, :3] == 3).all() and (y[:, 3 + k:] == 3).all()
        z = x.contiguous()
        want = cr.block_norm(z, cr.Norm("layer"))
        assert torch.equal(cr.block_norm(z, cr.Norm("layer"), out=z), want)


def test_empty_calls():
    x = torch.empty(0, 64, device="cuda")
    assert cr.block_norm(x, cr.Norm("rms")).shape == (0, 64)
    h, y = cr.block_update(x, x, norm=cr.Norm("rms"))
    assert h.shape == y.shape == (0, 64)
