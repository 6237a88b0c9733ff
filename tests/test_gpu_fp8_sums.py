"""How exact the sums of the FP8 linears are, value by value (GPU).

float32 outputs: products are exact and added in float32.

bfloat16 outputs come from the FP8 instruction.  It cuts the products of 8 consecutive features to a
multiple of 2^(e - 13), e the largest sum of two factors' exponents among the 8 (an E4M3 subnormal's
exponent, and a zero's at most, is -6), and adds those 8 exactly and the rest in float32.  The product
that has e keeps all of its 6 fraction bits, the other 7 lose less than one unit each: 7 U in all, U
the sum of the groups' units times their scales.  The float32 additions are off by at most
(k + 2) 2^-23 S, S = sum |x w| + |bias|, as in test_gpu_fp8.py; GELU has a slope of at most 1.13 and
its polynomial is off by 3.3e-7 max(1, |y|); the output's rounding is at most 2^-8 of the value.

Sums that cancel: where every product and every partial sum is a whole number below 2^23 and no group
of 8 holds products more than 2^13 apart, all of it is exact, whatever size the blocks before had.
"""

import pytest
import torch

import block_reference as ref
import hadamard_rotated_int8_amd as cr

pytestmark = pytest.mark.gpu

E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    cr.lib()
    yield
    torch.cuda.synchronize()


def _codes(q):
    return q.float().double()


def _row_scales(x, rows):
    return x.scale[rows].float().double()  # [rows, kb]


def _weight_scales(w, cols):
    return w.scale.float().double().repeat_interleave(128, 0)[:w.q.shape[0]][cols]  # [cols, kb]


def _exponents(v):
    return torch.where(v == 0, torch.full_like(v, -6), (torch.frexp(v).exponent - 1).double()).clamp_min(-6)


def _check(y, x, w, gelu, out):
    """y against the codes' exact sums: every row and column at the ends, a stride of those between."""
    m, k = x.q.shape
    n = w.q.shape[0]

    def some(size):
        at = set(range(min(size, 9))) | set(range(max(size - 9, 0), size)) | set(range(0, size, max(size // 12, 1)))
        return torch.tensor(sorted(at), device="cuda")

    rows, cols = some(m), some(n)
    sx, sw = _row_scales(x, rows), _weight_scales(w, cols)
    qx, qw = _codes(x.q[rows]), _codes(w.q[cols])
    bias = torch.zeros(len(cols), device="cuda", dtype=torch.float64) if w.bias is None else w.bias[cols].double()
    want, size, unit = bias.expand(len(rows), -1).clone(), bias.abs().expand(len(rows), -1).clone(), 0
    for b in range(sx.shape[1]):
        f = slice(128 * b, min(128 * b + 128, k))
        s = sx[:, None, b] * sw[None, :, b]
        p = qx[:, None, f] * qw[None, :, f]
        want += s * p.sum(2)
        size += s * p.abs().sum(2)
        e = _exponents(qx[:, None, f]) + _exponents(qw[None, :, f])
        unit = unit + s * torch.exp2(e.view(*e.shape[:2], -1, 8).amax(3) - 13).sum(2)
    off = (k + 2) * 2.0 ** -23 * size + (7 * unit if out == torch.bfloat16 else 0)
    if gelu:
        off = 1.13 * off + 3.3e-7 * want.abs().clamp_min(1) + 2.0 ** -23 * want.abs()
        want = want * torch.special.ndtr(want)
    tol = off + (2.0 ** -8 * (want.abs() + off) if out == torch.bfloat16 else 0)
    over = (y[rows][:, cols].double() - want).abs() - tol
    assert bool((over <= 0).all()), (over.max().item(), (over > 0).sum().item())


def _uneven(m, k, g):
    """Features of very different size."""
    x = torch.randn(m, k, generator=g, device="cuda")
    return (x * torch.exp(2 * torch.randn(k, generator=g, device="cuda"))).to(torch.bfloat16)


def _spiky(m, k, g):
    """One value in eight is large, of either sign, and the others just at the edge of what is kept."""
    large = torch.rand(m, k, generator=g, device="cuda") < 0.125
    sign = torch.sign(torch.randn(m, k, generator=g, device="cuda"))
    small = 1 + torch.randint(0, 8, (m, k), generator=g, device="cuda") / 8
    return torch.where(large, 256 * sign, small * torch.exp2(torch.randint(0, 3, (m, k), generator=g,
                                                                           device="cuda").float()))


# rows as they are, tiles of few rows, of middle sizes, large tiles (256 x 256, or 256 x 128 with
# float32 weight scales: sizes for both kinds), whole and ragged, several to a workgroup
SIZES = [(3, 300, 1296), (40, 200, 1296), (333, 1000, 2064), (2113, 2100, 656), (4100, 3900, 1296),
         (4000, 3900, 1296), (1700, 3900, 656), (130, 65000, 528)]


@pytest.mark.parametrize("f32", [False, True], ids=["e8m0", "f32scale"])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("gelu", [False, True], ids=["", "gelu"])
@pytest.mark.parametrize("data", [_uneven, _spiky])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_every_value_is_within_its_bound(m, n, k, data, gelu, out, f32):
    print(f"[gpu] fp8 linear by value {m}x{n}x{k} {data.__name__} {out} gelu={gelu} f32scale={f32}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(m + n)
    x = data(m, k, g)
    w = cr.fp8_quantize_weights(torch.randn(n, k, generator=g, device="cuda") * 0.02 if data is _uneven else
                                data(n, k, g).abs(), torch.randn(n, generator=g, device="cuda"))
    if data is _spiky:  # sums of order one
        w.scale = (w.scale.float() * 2.0 ** -14).to(E8M0)
    if f32:
        w.scale = w.scale.float() * (1 + torch.rand(w.scale.shape, generator=g, device="cuda"))
    y = cr.fp8_linear(x, w, out_dtype=out, gelu=gelu)
    _check(y, cr.fp8_pack_activations(x), w, gelu, out)


@pytest.mark.parametrize("f32,m,n,k", [(False, 4200, 4200, 16640), (True, 4000, 4000, 33024)],
                         ids=["e8m0", "f32scale"])
def test_large_outputs_of_very_long_rows(f32, m, n, k):
    """More blocks of features than a workgroup has threads to fetch their weight scales at once, several
    tiles to a workgroup: small integers, exact."""
    print(f"[gpu] fp8 linear large and long {m}x{n}x{k} f32scale={f32}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(k)
    kb, nb = k // 128, -(-n // 128)

    def integers(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device="cuda")

    x = cr.Fp8Activation(integers(-3, 4, m, k).float().to(E4M3),
                         integers(127, 129, kb, m).to(torch.uint8).view(E8M0).t())
    scale = 1 + 0.5 * integers(0, 2, nb, kb).float() if f32 else integers(127, 129, nb, kb).to(torch.uint8).view(E8M0)
    w = cr.Fp8Weights(integers(-2, 3, n, k).float().to(E4M3), scale, integers(-8, 9, n).float())
    y = cr.fp8_linear(x, w, out_dtype=torch.bfloat16)
    want = w.bias.double().expand(m, -1).clone()
    step = 1024
    for at in range(0, k, step):  # (whole blocks, in pieces that fit)
        f, b = slice(at, min(at + step, k)), slice(at // 128, -(-min(at + step, k) // 128))
        d = _codes(x.q[:, f]) * x.scale.float().double()[:, b].repeat_interleave(128, 1)
        v = _codes(w.q[:, f]) * _weight_scales(w, slice(None))[:, b].repeat_interleave(128, 1)
        want += d @ v.t().contiguous()
    assert want.abs().max() < 2 ** 22  # (in halves: exact in float32)
    assert torch.equal(y, want.float().to(torch.bfloat16))


@pytest.mark.parametrize("f32", [False, True], ids=["e8m0", "f32scale"])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("m,n,k", [(3, 300, 5136), (40, 200, 5136), (333, 1000, 5136), (4100, 3900, 5136), (4000, 3900, 5136)])
def test_large_blocks_that_cancel_leave_the_small_ones(m, n, k, out, f32):
    """The first block holds one product of 2^p, the last one its opposite; small integers between."""
    print(f"[gpu] fp8 linear cancelling blocks {m}x{n}x{k} {out} f32scale={f32}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(n)
    kb, nb = -(-k // 128), -(-n // 128)
    last = 128 * (kb - 1)
    for p in (14, 17, 20):
        x = torch.randint(-3, 4, (m, k), generator=g, device="cuda").float()
        x[:, :128], x[:, last:] = 0, 0
        x[:, 5], x[:, last + 3] = 2.0 ** p, -(2.0 ** p)
        q = torch.randint(-2, 3, (n, k), generator=g, device="cuda").float()
        q[:, 5], q[:, last + 3] = 1, 1
        ones = torch.ones(nb, kb, device="cuda") if f32 else \
            torch.full((nb, kb), 127, dtype=torch.uint8, device="cuda").view(E8M0)
        w = cr.Fp8Weights(q.to(E4M3), ones)
        # (the pack is exact: blocks of one value or of small integers)
        want = x.double() @ q.double().t().contiguous()
        assert want.abs().max() < 2 ** 14 and want.norm() > 0
        assert torch.equal(cr.fp8_linear(x, w, out_dtype=out), want.float().to(out)), p


@pytest.mark.parametrize("m,n,k", [(4000, 3900, 400), (6100, 4090, 400), (8190, 2040, 528), (255, 65000, 400)])
def test_large_outputs_with_float32_scales(m, n, k):
    """More ragged edges of the 256 x 128 tiles, with rows that allow wide stores and rows that do not:
    small integers, exact, and nothing beside the outputs."""
    print(f"[gpu] fp8 linear large float32 scales {m}x{n}x{k}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(n)
    kb, nb = -(-k // 128), -(-n // 128)

    def integers(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device="cuda")

    x = cr.Fp8Activation(integers(-3, 4, m, k).float().to(E4M3),
                         integers(127, 129, kb, (m + 3) // 4 * 4).to(torch.uint8).view(E8M0).t()[:m])
    w = cr.Fp8Weights(integers(-2, 3, n, k).float().to(E4M3), 1 + 0.5 * integers(0, 2, nb, kb).float(),
                      integers(-8, 9, n).float())
    d = _codes(x.q) * x.scale.float().double().repeat_interleave(128, 1)[:, :k]
    v = _codes(w.q) * _weight_scales(w, slice(None)).repeat_interleave(128, 1)[:, :k]
    want = (d @ v.t().contiguous() + w.bias.double()).float().to(torch.bfloat16)
    assert torch.equal(cr.fp8_linear(x, w, out_dtype=torch.bfloat16), want)
    wide = torch.full((m, n + 11), 7.0, dtype=torch.bfloat16, device="cuda")
    for at in (1, 8):
        cr.fp8_linear(x, w, out=wide[:, at:at + n])
        assert torch.equal(wide[:, at:at + n], want)
        assert (wide[:, :at] == 7).all() and (wide[:, at + n:] == 7).all()
        wide.fill_(7)
