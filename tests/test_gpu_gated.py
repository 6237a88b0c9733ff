"""The gated pair of projections and its way back, against plain 64-bit references (GPU).

* A projection's sum, from the codes' exact values: float32 outputs (k + 2) 2^-23 S, S = sum |x w| +
  |bias|; with bfloat16 outputs the FP8 instruction loses besides less than 7 2^-13 of the largest
  product of each 8 neighbouring features (include/convrot.h), which is at most 7 2^-13 S.
* y = act(G) U: with |act'| <= 1.13, 1.13 |U| dG + |act(G)| dU (and 1.13 dG dU), SiLU within 2^-21 of
  its value (an exponential, a sum and a reciprocal, a unit each), GELU within 3.3e-7 max(1, |G|), the
  product's rounding 2^-24, the output's 2^-8 or 2^-24.
* Gradients at the projections are float32 expressions of given values: relative errors of a few units
  in each factor, 2^-20 together of s (1 + |g| (1 - s)) or (Phi + |g| phi) (1 + g^2), and one rounding.
"""

import ctypes
import math

import pytest
import torch

import block_reference as ref
import hadamard_rotated_int8_amd as cr
from hadamard_rotated_int8_amd import block as impl

pytestmark = pytest.mark.gpu

E8M0 = torch.float8_e8m0fnu
BF16, F32 = torch.bfloat16, torch.float32


def _weights(n, k, scale, seed, bias=True):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(n, k, generator=g) * 0.05 * torch.exp(torch.randn(n, 1, generator=g) * 0.3)
    b = (torch.randn(n, generator=g) * 0.1).cuda() if bias else None
    out = cr.fp8_quantize_weights(w.cuda(), b)
    if scale == F32:  # any scales: those of the powers of two, times a factor for each block
        factor = 0.5 + torch.rand(out.scale.shape, generator=g)
        out = cr.Fp8Weights(out.q, out.scale.float() * factor.cuda(), b)
    return out


def _x(m, k, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(m, k, generator=g) * torch.exp(0.7 * torch.randn(k, generator=g))).to(dtype).cuda()


def _dequantised(w):
    n, k = w.q.shape
    s = w.scale.float().double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    return w.q.float().double() * s


def _act(v, act):
    return v * torch.sigmoid(v) if act == "silu" else v * torch.special.ndtr(v)


def _sums(xd, w, exact):
    """A projection of dequantised rows in 64 bits, and how far the kernel's may be from it."""
    wd = _dequantised(w)
    k = xd.shape[1]
    v, size = xd @ wd.t(), xd.abs() @ wd.abs().t()
    if w.bias is not None:
        v, size = v + w.bias.double(), size + w.bias.double().abs()
    return v, size * ((k + 2) * 2.0 ** -23 + (0 if exact else 7 * 2.0 ** -13))


def _sharp(xd, w, rows, cols):
    """_sums for some rows and columns, with the instruction's loss by groups of 8."""
    wd = _dequantised(w)[cols]
    p = xd[rows][:, None] * wd[None]
    k = p.shape[2]
    top = p.abs().view(*p.shape[:2], k // 8, 8).amax(3).sum(2)
    v, size = p.sum(2), p.abs().sum(2)
    if w.bias is not None:
        b = w.bias.double()[cols]
        v, size = v + b, size + b.abs()
    return v, (k + 2) * 2.0 ** -23 * size + 7 * 2.0 ** -13 * top


def _product(g, dg, u, du, act, dtype):
    """act(G) U and its bound from the projections and theirs."""
    a = _act(g, act)
    da = 1.13 * dg + (2.0 ** -21 * a.abs() if act == "silu" else 3.3e-7 * g.abs().clamp_min(1))
    y = a * u
    tol = da * u.abs() + (a.abs() + da) * du + 2.0 ** -23 * y.abs()
    return y, tol + (y.abs() + tol) * torch.finfo(dtype).eps / 2 + 1e-37


def _close(got, want, tol):
    off = (got.double() - want).abs()
    assert not got.isnan().any() and (off <= tol).all(), ((off - tol).max().item(), off.max().item())


def _check(x, gate, up, act, dtype, y, kept):
    p = x if isinstance(x, cr.Fp8Activation) else cr.fp8_pack_activations(x)
    m, k = p.q.shape
    n = gate.q.shape[0]
    xd = p.q.float().double() * p.scale.float().double().repeat_interleave(128, 1)[:, :k]
    g, dg = _sums(xd, gate, dtype == F32)
    u, du = _sums(xd, up, dtype == F32)
    assert y.shape == (m, n) and y.dtype == dtype
    _close(y, *_product(g, dg, u, du, act, dtype))
    if kept is not None:
        for t, v, dv in ((kept[0], g, dg), (kept[1], u, du)):
            assert t.dtype == BF16 and t.shape == (m, n)
            _close(t, v, dv + (v.abs() + dv) * 2.0 ** -8)
    if dtype == BF16:
        some = lambda size: torch.tensor(sorted(  # noqa: E731
            set(range(min(size, 5))) | set(range(max(size - 5, 0), size)) | set(range(0, size, max(size // 9, 1)))))
        rows, cols = some(m).cuda(), some(n).cuda()
        (g, dg), (u, du) = _sharp(xd, gate, rows, cols), _sharp(xd, up, rows, cols)
        _close(y[rows][:, cols], *_product(g, dg, u, du, act, dtype))


SCALES = pytest.mark.parametrize("scale", [E8M0, F32], ids=["e8m0", "f32"])
DTYPES = pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])


@SCALES
@DTYPES
@pytest.mark.parametrize("m, k, n", [
    # a few rows as they are
    (1, 16, 1), (1, 128, 16), (1, 1040, 333), (3, 4112, 17), (16, 2048, 4104), (7, 400, 33),
    # packed: tiles of one to four groups of waves, one workgroup to a CU, two
    (17, 16, 1), (33, 144, 9), (40, 2048, 1500), (64, 1024, 5000), (100, 512, 1000), (129, 1040, 2056),
    (200, 4112, 700), (333, 640, 4104), (500, 384, 3000), (1000, 256, 2001),
    # many tiles
    (1024, 512, 8192), (1100, 400, 8200), (1030, 1168, 8323), (2048, 384, 4097)])
def test_sizes(m, k, n, dtype, scale):
    gate, up = _weights(n, k, scale, n + k), _weights(n, k, scale, n + k + 1, bias=n % 2 == 0)
    for act, keep in (("silu", True), ("gelu", False)):
        x = _x(m, k, BF16 if keep else F32, m + k)
        got = cr.fp8_gated(x, gate, up, act=act, out_dtype=dtype, keep=keep)
        y, kept = got if keep else (got, None)
        _check(x, gate, up, act, dtype, y, kept)


@SCALES
@pytest.mark.parametrize("m, k, n", [(2, 256, 40), (100, 256, 512), (1024, 512, 8192)])
def test_activations_and_outputs(m, k, n, scale):
    gate, up = _weights(n, k, scale, 1), _weights(n, k, scale, 2)
    x = _x(m, k, F32, 3)
    p = cr.fp8_pack_activations(x)
    want = cr.fp8_gated(p, gate, up, out_dtype=BF16)
    _check(p, gate, up, "silu", BF16, want, None)
    y, kept = cr.fp8_gated(p, gate, up, out_dtype=BF16, keep=True)
    assert torch.equal(y, want)
    for pad in (3, 8):  # rows that allow no vector stores, and rows that do
        wide = torch.full((m, n + 2 * pad), 7.0, dtype=BF16, device="cuda")
        out = wide[:, pad:pad + n]
        assert cr.fp8_gated(p, gate, up, out=out) is out
        assert torch.equal(out, want)
        assert (wide[:, :pad] == 7).all() and (wide[:, pad + n:] == 7).all()


def test_an_output_over_x():
    k = n = 512
    gate, up = _weights(n, k, E8M0, 1), _weights(n, k, E8M0, 2)
    for m in (5, 200):
        x = _x(m, k, F32, 3)
        want = cr.fp8_gated(cr.fp8_pack_activations(x), gate, up)
        assert torch.equal(cr.fp8_gated(x, gate, up, out=x), want)


def test_small_integers_are_exact():
    # every product and sum is a small integer; a gate of 30 makes act the identity to float32
    g = torch.Generator().manual_seed(0)
    for m, k, n in ((3, 256, 40), (70, 256, 130), (1024, 384, 8192)):
        x = torch.randint(-2, 3, (m, k), generator=g).float().cuda()
        x[:, 0] = 1.0
        wg, wu = torch.zeros(n, k), torch.randint(-2, 3, (n, k), generator=g).float()
        wg[:, 0] = 32.0
        gate, up = cr.fp8_quantize_weights(wg.cuda()), cr.fp8_quantize_weights(wu.cuda())
        want = 32.0 * (x.double() @ wu.cuda().double().t())
        y, kept = cr.fp8_gated(x, gate, up, out_dtype=F32, keep=True)
        assert torch.equal(y.double(), want)
        y2, kept2 = cr.fp8_gated(x, gate, up, act="gelu", out_dtype=BF16, keep=True)
        for a in (kept, kept2):
            assert (a[0] == 32.0).all() and torch.equal(a[1], (want / 32).to(BF16))
        assert torch.equal(y2, want.to(BF16))


def _nan_blocks(m, k, n):
    x = torch.ones(m, k)
    x[m // 2, k - 1] = math.nan
    gate, up = _weights(n, k, E8M0, 1), _weights(n, k, E8M0, 2)
    return x.cuda(), gate, up


@pytest.mark.parametrize("m, n", [(5, 40), (100, 500), (1024, 8192)])
def test_a_nan_stays_in_its_row(m, n):
    x, gate, up = _nan_blocks(m, 400, n)
    for dtype in (BF16, F32):
        y = cr.fp8_gated(x, gate, up, out_dtype=dtype)
        bad = y.isnan()
        assert bad[m // 2].all() and bad.sum() == n


# ---------------------------------------------------------------------------
# The way back
# ---------------------------------------------------------------------------

def _kept(m, n, seed, dtype=BF16):
    g = torch.Generator().manual_seed(seed)
    dy = (torch.randn(m, n, generator=g) * 1e-2).to(dtype).cuda()
    return dy, tuple((2.5 * torch.randn(m, n, generator=g)).to(BF16).cuda() for _ in range(2))


def _projection_gradients(dy, kept, act):
    """(dG, its float32 bound), (dU, its) in 64 bits."""
    dy, g, u = dy.double(), kept[0].double(), kept[1].double()
    if act == "silu":
        s = torch.sigmoid(g)
        a, slope, size = g * s, s * (1 + g * (1 - s)), s * (1 + g.abs() * (1 - s))
    else:
        # (torch.special.ndtr takes 1 + erf there and is off by 1 % at -7.8, in 64 bits)
        cdf, pdf = 0.5 * torch.special.erfc(-g * math.sqrt(0.5)), torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
        a, slope, size = g * cdf, cdf + g * pdf, (cdf + g.abs() * pdf) * (1 + g * g)
        # Below zero Phi(g) = erfc(x) / 2, x = -g / sqrt 2, and d ln erfc / d ln x is within 1 + 2 x^2 = 1 + g^2
        # of zero: x's two roundings (the constant's, the product's: 2^-23) come back as (1 + g^2) 2^-23
        # of Phi, as the density's exponent of g^2 / 2 makes them of the density.
        a_size = 1 + g * g
    if act == "silu":
        a_size = 1
    return ((dy * u * slope, 2.0 ** -20 * (dy * u).abs() * size + 1e-37),
            (dy * a, 2.0 ** -20 * (dy * a).abs() * a_size + 1e-37))


def _packed_gradients(dy, kept, act):
    """The FP8 activation that the library makes of both gradients."""
    m, n = dy.shape
    packed = impl._new_activation(m, 2 * impl._blocks(n) * 128, dy.device)
    outs = [torch.empty(m, n, dtype=BF16, device="cuda") for _ in range(2)]
    pk = impl._writable(impl._pack_args(packed))
    impl._launch(cr.lib().convrot_fp8_gated_backward, "convrot_fp8_gated_backward", dy.device,
                 impl._GATED_BACKWARD.pack(dy.data_ptr(), kept[0].data_ptr(), kept[1].data_ptr(), outs[0].data_ptr(),
                                           outs[1].data_ptr(), ctypes.addressof(pk), m, n, dy.stride(0),
                                           kept[0].stride(0), n, impl._DTYPE[dy.dtype], impl._gated_act(act)))
    return packed, outs


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("m, n", [(1, 1), (3, 16), (5, 130), (70, 1000), (33, 2049), (1, 13824), (300, 256)])
def test_projection_gradients(m, n, dtype, act):
    dy, kept = _kept(m, n, m + n, dtype)
    kept[0][0, 0] = -200.0  # both ends of the activation
    kept[0][m - 1, n - 1] = 200.0
    grads = _projection_gradients(dy, kept, act)
    packed, outs = _packed_gradients(dy, kept, act)
    for out, (want, tol) in zip(outs, grads):
        _close(out, want, tol + (want.abs() + tol) * 2.0 ** -8)
    # The codes: nearest to a value within the bound, of the block's least power of two
    np = impl._blocks(n) * 128
    for i, (want, tol) in enumerate(grads):
        q = packed.q[:, i * np:(i + 1) * np].float().double().cpu()
        s = packed.scale[:, i * np // 128:(i + 1) * np // 128].float().double().cpu()
        assert (q[:, n:] == 0).all()
        want, tol = want.cpu(), tol.cpu()
        lo, hi = ref.pack((want.abs() - tol).clamp_min(0))[1], ref.pack(want.abs() + tol)[1]
        byte = packed.scale[:, i * np // 128:(i + 1) * np // 128].contiguous().view(torch.uint8).cpu()
        zero = (want.abs() - tol).clamp_min(0) == 0
        blocks = torch.nn.functional.pad(zero, (0, np - n), value=True).view(m, -1, 128).all(2)
        assert ((byte >= lo) | blocks).all() and ((byte <= hi) | blocks).all()
        each = s.repeat_interleave(128, 1)[:, :n]
        step = torch.maximum(torch.ldexp(torch.ones_like(want), torch.frexp(want.abs() / each).exponent - 4),
                             torch.tensor(2.0 ** -9, dtype=torch.float64))
        assert ((q[:, :n] * each - want).abs() <= step * each / 2 * 1.001 + tol).all()


@SCALES
@pytest.mark.parametrize("m, k, n", [(1, 16, 1), (5, 400, 130), (70, 1040, 1000), (33, 144, 2049), (1030, 1024, 1500),
                                     (4100, 4336, 200)])
def test_gradient_at_x(m, k, n, scale):
    gate, up = _weights(n, k, scale, 1), _weights(n, k, scale, 2)
    back = cr.fp8_transpose_weights([gate, up])
    np = impl._blocks(n) * 128
    assert back.q.shape == (k, 2 * np)
    wd = _dequantised(back)
    assert torch.equal(wd[:, :n], _dequantised(gate).t()) and torch.equal(wd[:, np:np + n], _dequantised(up).t())
    assert (wd[:, n:np] == 0).all() and (wd[:, np + n:] == 0).all()
    if m > 4096 and torch.cuda.get_device_properties(0).multi_processor_count == 256:
        assert impl._whole_rounds(m, back, torch.device("cuda", 0)) == 3840  # two products
    dy, kept = _kept(m, n, m + n)
    packed, outs = _packed_gradients(dy, kept, "silu")
    dx, grads = cr.fp8_gated_backward(dy, kept, back)
    assert dx.dtype == BF16 and dx.shape == (m, k)
    assert all(torch.equal(a, b) for a, b in zip(outs, grads))
    d = packed.q.float().double() * packed.scale.float().double().repeat_interleave(128, 1)
    want, size = d @ wd.t(), d.abs() @ wd.abs().t()
    tol = size * ((2 * np + 2) * 2.0 ** -23 + 7 * 2.0 ** -13)
    _close(dx, want, tol + (want.abs() + tol) * 2.0 ** -8 + 1e-37)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradient_at_x_against_differences(act):
    # of f(X) = sum dY act(X Wg^T + bg) (X Wu^T + bu) in 64 bits; the packed gradients are off by 2^-4
    # of each (or of their block's smallest step, 2^-10 2^-8 of its largest)
    m, k, n = 4, 48, 200
    gate, up = _weights(n, k, E8M0, 5), _weights(n, k, E8M0, 6)
    x = cr.fp8_pack_activations(_x(m, k, F32, 7))
    xd = x.q.float().double() * x.scale.float().double().repeat_interleave(128, 1)[:, :k]
    y, kept = cr.fp8_gated(x, gate, up, act=act, keep=True)
    dy = _kept(m, n, 8, F32)[0]
    dx, (dg, du) = cr.fp8_gated_backward(dy, kept, cr.fp8_transpose_weights([gate, up]), act=act)
    wg, wu = _dequantised(gate), _dequantised(up)

    def f(v):
        return (dy.double() * _act(v @ wg.t() + gate.bias.double(), act) * (v @ wu.t() + up.bias.double())).sum(1)

    h = 1e-5
    diff = torch.stack([(f(xd + h * e) - f(xd - h * e)) / (2 * h)
                        for e in torch.eye(k, dtype=torch.float64, device="cuda")], dim=1)
    tol = torch.zeros_like(diff)
    for d, w in ((dg, wg), (du, wu)):
        d = d.double().abs()
        top = torch.nn.functional.pad(d, (0, 56)).view(m, 2, 128).amax(2).repeat_interleave(128, 1)[:, :n]
        # (a code's half step; the kept values' own rounding moves act, its slope and U by 2^-8 of theirs
        #  and, the slope's slope being at most 1, |G| 2^-8 of dY U)
        each = 2.0 ** -4 * d + 2.0 ** -17 * top + 2.0 ** -7 * d
        if w is wg:
            each = each + 2.0 ** -8 * (kept[0].double() * dy.double() * kept[1].double()).abs()
        tol += each @ w.abs()
    assert ((dx.double() - diff).abs() <= 1.05 * tol + 2.0 ** -8 * diff.abs() + 1e-8).all()
    assert (dx.double() - diff).norm() <= 0.05 * diff.norm()


def test_backward_strides_and_empty_rows():
    m, k, n = 9, 144, 100
    gate, up = _weights(n, k, E8M0, 1), _weights(n, k, E8M0, 2)
    back = cr.fp8_transpose_weights([gate, up])
    dy, kept = _kept(m, n, 3)
    want = cr.fp8_gated_backward(dy, kept, back)
    both = torch.cat(kept, dim=1)
    wide = torch.cat([dy, dy], dim=1)[:, n - 1:2 * n - 1].clone()
    wide = torch.nn.functional.pad(dy, (1, 2))
    got = cr.fp8_gated_backward(wide[:, 1:n + 1], (both[:, :n], both[:, n:]), back)
    assert torch.equal(got[0], want[0]) and all(torch.equal(a, b) for a, b in zip(got[1], want[1]))
    dx, grads = cr.fp8_gated_backward(dy[:0], tuple(t[:0] for t in kept), back)
    assert dx.shape == (0, k) and grads[0].shape == (0, n)
    y, kept = cr.fp8_gated(torch.empty(0, k, device="cuda"), gate, up, keep=True)
    assert y.shape == (0, n) and kept[1].shape == (0, n)


@pytest.mark.parametrize("m, k, n", [(1, 1024, 3000), (100, 512, 512), (1024, 512, 8192)])
def test_graphs_and_streams(m, k, n):
    gate, up = _weights(n, k, E8M0, 1), _weights(n, k, E8M0, 2)
    back = cr.fp8_transpose_weights([gate, up])
    x, dy = _x(m, k, BF16, 1), _kept(m, n, 2)[0]

    def step():
        y, kept = cr.fp8_gated(x, gate, up, out_dtype=BF16, keep=True)
        dx, grads = cr.fp8_gated_backward(dy, kept, back)
        return [y, *kept, dx, *grads]

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res = step()
        graphs.append((graph, res))
    for round in range(3):
        x.copy_(_x(m, k, BF16, 20 + round))
        dy.copy_(_kept(m, n, 30 + round)[0])
        eager = step()
        for graph, res in graphs:
            for t in res:
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(res, eager))


def test_refusals():
    k, n = 128, 64
    gate, up = _weights(n, k, E8M0, 1), _weights(n, k, E8M0, 2)
    other, f32 = _weights(n + 1, k, E8M0, 3), _weights(n, k, F32, 4)
    x = _x(20, k, F32, 1)
    for args, kw in [((x, gate, other), {}), ((x, gate, f32), {}), ((x, gate, up), dict(act="relu")),
                     ((x, gate, up), dict(out_dtype=torch.float16)),
                     ((x, gate, up), dict(out=torch.empty(20, n + 1, device="cuda"))),
                     ((x.cpu(), gate, up), {})]:
        with pytest.raises(ValueError):
            cr.fp8_gated(*args, **kw)
    with pytest.raises(cr.ConvrotError):
        cr.fp8_gated(x[:, :112].contiguous(), gate, up)  # k does not fit
    back = cr.fp8_transpose_weights([gate, up])
    dy, kept = _kept(20, n, 1)
    for args in [(dy[:, 1:], kept, back), (dy, kept[:1], back), (dy, (kept[0], kept[1].float()), back),
                 (dy, kept, gate), (dy, (kept[0], kept[1].t().contiguous().t()), back)]:
        with pytest.raises(ValueError):
            cr.fp8_gated_backward(*args)
    with pytest.raises(ValueError):
        cr.fp8_transpose_weights([gate, f32])
    with pytest.raises(ValueError):
        cr.fp8_transpose_weights([])
