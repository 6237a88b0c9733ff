"""FP8 linears with a scale for each block of 128, against plain 64-bit references (GPU).

* Codes and scales are exact: powers of two make the division exact, so every
  code is the E4M3 value nearest to an exact quotient.
* Small integers: every product and sum is a small integer times a power of
  two, exact in any order and format, so outputs are equal bit for bit (each
  bfloat16 output is the rounding of the exact value).
* Random values, float32 output: products are exact, the K - 1 additions of a
  sum are off by at most 2^-23 of the running sum each (the matrix cores may
  truncate), and the bias and its addition by one more: (K + 2) 2^-23 S with
  S = sum |x w| + |bias|.
* Random values, bfloat16 output: the rounding is at most 2^-8 of each value
  (8 significant bits: a step of 2^-7 of the power of two below, half of it),
  and the FP8 instruction's dropped low product bits
  are within 2^-13 of the result in the 2-norm (they are 4e-5 = 2^-14.6 of it
  for the most uneven inputs measured), so 2^-8 + 2^-13 in the 2-norm.
* GELU has a slope of at most 1.13 and its polynomial is off by at most
  3.3e-7 max(1, |y|).
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


def _bytes(t):
    return t.contiguous().view(torch.uint8).cpu().int()


def _inputs(m, k, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(m, k, generator=g) * torch.exp(2 * torch.randn(k, generator=g))
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,k", [(1, 16), (3, 128), (1, 144), (257, 1040), (70, 4112), (5, 20000)])
def test_pack_is_exact(m, k, dtype):
    print(f"[gpu] fp8 pack {m}x{k} {dtype}", flush=True)
    x = _inputs(m, k, dtype, m + k)
    p = cr.fp8_pack_activations(x.cuda())
    d, byte = ref.pack(x)
    assert torch.equal(_bytes(p.scale), byte.int())
    assert torch.equal(ref.dequantised_rows(p.q, p.scale), d)


def _edge_rows():
    """Rows of one block each with values where the scale or a code is decided."""
    rows = []

    def row(*v):
        r = torch.zeros(128)
        r[:len(v)] = torch.tensor(v, dtype=torch.float64).float()
        rows.append(r)

    nxt = torch.nextafter(torch.tensor(448.0), torch.tensor(1e9)).item()
    row(448.0, 447.0, -448.0)
    row(nxt, 1.0)                       # the next scale
    row(448.0 * 2.0 ** -20, 1e-9)
    row(256.0, 17.0, 19.0, 21.0, -17.0)  # ties between codes
    row(256.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -10 * 1.0000001)  # E4M3 subnormals and their ties
    row(*([0.0] * 128))
    row(-0.0, 0.0)
    row(1e-45, -3e-45)                  # float32 subnormals: the scale's lower end
    row(2.0 ** -126)
    row(2.0 ** -118, 2.0 ** -130)
    row(3.4028234663852886e38, -1.0)
    row(2.0 ** 127, 2.0 ** 119)
    return torch.stack(rows)


def test_pack_edges():
    x = _edge_rows()
    p = cr.fp8_pack_activations(x.cuda())
    d, byte = ref.pack(x)
    assert torch.equal(_bytes(p.scale), byte.int())
    assert torch.equal(ref.dequantised_rows(p.q, p.scale), d)


def test_pack_blocks_that_are_not_finite():
    x = torch.ones(3, 384)
    x[0, 130] = float("inf")
    x[1, 383] = float("nan")
    x[2, 0] = float("-inf")
    p = cr.fp8_pack_activations(x.cuda())
    d, byte = ref.pack(x)
    assert torch.equal(_bytes(p.scale), byte.int())
    got = ref.dequantised_rows(p.q, p.scale)
    assert torch.equal(torch.isnan(got), torch.isnan(d))
    assert torch.equal(got.nan_to_num(7.0), d.nan_to_num(7.0))
    w = cr.fp8_quantize_weights(torch.ones(16, 384).cuda())
    for dt in (torch.float32, torch.bfloat16):
        assert torch.isnan(cr.fp8_linear(p, w, out_dtype=dt)).all()  # every row holds such a block


def test_pack_strided_rows_and_given_output():
    wide = _inputs(40, 512, torch.bfloat16, 5).cuda()
    x = wide[::2, 64:64 + 272]  # row stride 1024, an offset of 128 bytes
    q = torch.full((20, 272), 1, dtype=torch.uint8).cuda().view(E4M3)
    s = torch.full((3, 32), 9, dtype=torch.uint8).cuda()
    out = cr.Fp8Activation(q, s.view(E8M0).t()[8:28])
    assert cr.fp8_pack_activations(x, out) is out
    d, byte = ref.pack(x.cpu())
    assert torch.equal(_bytes(out.scale), byte.int())
    assert torch.equal(ref.dequantised_rows(out.q, out.scale), d)
    assert (s[:, :8] == 9).all() and (s[:, 28:] == 9).all()  # nothing beside the scales
    # rows 4 .. 17 of it are an activation of their own
    w = cr.fp8_quantize_weights(torch.randn(40, 272).cuda())
    part = cr.fp8_linear(cr.Fp8Activation(out.q[4:18], out.scale[4:18]), w)
    assert torch.equal(part, cr.fp8_linear(out, w)[4:18])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,k", [(1, 16), (128, 128), (130, 400), (300, 1040)])
def test_weight_quantisation_is_exact(n, k, dtype):
    print(f"[gpu] fp8 weights {n}x{k} {dtype}", flush=True)
    w = _inputs(n, k, dtype, n * k)
    W = cr.fp8_quantize_weights(w.cuda())
    d, byte = ref.quantize(w)
    assert torch.equal(_bytes(W.scale), byte.int())
    assert torch.equal(ref.dequantised_weights(W.q, W.scale), d)


def _integers(m, n, k, f32, seed, sign_only=False):
    """An activation and weights of small integers with scales of 1 and 2 (or 1 and 1.5)."""
    g = torch.Generator().manual_seed(seed)
    kb, nb = -(-k // 128), -(-n // 128)
    qx = torch.randint(-3, 4, (m, k), generator=g).float().to(E4M3).cuda()
    qw = torch.randint(-2, 3, (n, k), generator=g).float().to(E4M3).cuda()
    sx = torch.randint(127, 129, (kb, (m + 3) // 4 * 4), generator=g).to(torch.uint8).cuda()
    if f32:
        sw = (1 + 0.5 * torch.randint(0, 2, (nb, kb), generator=g)).float().cuda()
    else:
        sw = torch.randint(127, 129, (nb, kb), generator=g).to(torch.uint8).view(E8M0).cuda()
    bias = torch.randint(-8, 9, (n,), generator=g).float().cuda()
    return cr.Fp8Activation(qx, sx.view(E8M0).t()[:m]), cr.Fp8Weights(qw, sw, bias)


SHAPES = [(1, 1, 16), (2, 33, 5136), (17, 100, 656), (31, 64, 4112), (32, 31, 128), (40, 257, 1040), (64, 300, 2064), (65, 64, 640), (1, 128, 128), (2, 130, 144), (7, 64, 400), (15, 300, 1040), (16, 640, 2048),
          (17, 96, 128), (33, 257, 272), (64, 128, 640), (100, 1000, 1296), (129, 129, 384),
          (256, 512, 512), (300, 770, 912), (513, 260, 528), (1, 4096, 5120), (5, 1500, 13824),
          (17, 8500, 144), (40, 4200, 272), (64, 4096, 400)]


@pytest.mark.parametrize("f32", [False, True], ids=["e8m0", "f32scale"])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_linear_small_integers(m, n, k, out, f32):
    print(f"[gpu] fp8 linear integers {m}x{n}x{k} {out} f32scale={f32}", flush=True)
    x, w = _integers(m, n, k, f32, m + 3 * n + k)
    y = cr.fp8_linear(x, w, out_dtype=out)
    want = ref.dequantised_rows(x.q, x.scale) @ ref.dequantised_weights(w.q, w.scale).t()
    want = want + w.bias.cpu().double()
    assert want.abs().max() < 2 ** 22  # (in quarters: exact in float32)
    assert torch.equal(y.cpu(), want.float().to(out))


@pytest.mark.parametrize("f32", [False, True], ids=["e8m0", "f32scale"])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("gelu", [False, True], ids=["", "gelu"])
@pytest.mark.parametrize("m,n,k,xt", [(1, 384, 2048, torch.bfloat16), (13, 200, 1040, torch.float32),
                                      (16, 96, 272, torch.bfloat16), (130, 520, 4112, torch.bfloat16),
                                      (700, 300, 1024, torch.float32)])
def test_linear_random(m, n, k, xt, gelu, out, f32):
    print(f"[gpu] fp8 linear {m}x{n}x{k} {xt}->{out} gelu={gelu} f32scale={f32}", flush=True)
    g = torch.Generator().manual_seed(m * n)
    x = _inputs(m, k, xt, k)
    W = cr.fp8_quantize_weights((torch.randn(n, k, generator=g) * 0.02).cuda(),
                                (torch.randn(n, generator=g)).cuda())
    if f32:
        W.scale = W.scale.float() * (1 + torch.rand(W.scale.shape, generator=g).cuda())
    y = cr.fp8_linear(x.cuda(), W, out_dtype=out, gelu=gelu)
    d, _ = ref.pack(x)
    w = ref.dequantised_weights(W.q, W.scale)
    want = d @ w.t() + W.bias.cpu().double()
    size = d.abs() @ w.abs().t() + W.bias.cpu().double().abs()
    tol = (k + 2) * 2.0 ** -23 * size
    if gelu:
        tol = 1.13 * tol + 3.3e-7 * want.abs().clamp_min(1) + 2.0 ** -23 * want.abs()
        slope, want = 1.13, ref.gelu(want)
    if out == torch.float32:
        assert ((y.cpu().double() - want).abs() <= tol).all()
    else:
        linear = d @ w.t() + W.bias.cpu().double()
        off = (y.cpu().double() - want).norm()
        assert off <= 2.0 ** -8 * want.norm() + (1.13 if gelu else 1.0) * 2.0 ** -13 * linear.norm()


@pytest.mark.parametrize("m", [1, 9, 200, 600])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_grouped_equals_single(m, out):
    """A grouped launch gives what each weight gives alone, into strided outputs whose surroundings
    stay as they were.

    The two may add in different orders (how the work is divided depends on all of a launch's
    outputs): each is within the module's tolerance of the exact sum, so they are within twice that of
    each other.
    """
    x = _inputs(m, 784, torch.bfloat16, m).cuda()
    g = torch.Generator().manual_seed(m)
    ws = [cr.fp8_quantize_weights((torch.randn(n, 784, generator=g) * 0.02).cuda(),
                                  torch.randn(n, generator=g).cuda() if n != 77 else None)
          for n in (300, 77, 0, 128)]
    p = cr.fp8_pack_activations(x)
    d = ref.dequantised_rows(p.q, p.scale)

    def check(a, b, w):
        a, b = a.cpu().double(), b.cpu().double()
        v = ref.dequantised_weights(w.q, w.scale)
        bias = torch.zeros(v.shape[0], dtype=torch.float64) if w.bias is None else w.bias.cpu().double()
        linear = d @ v.t() + bias
        if out == torch.float32:
            tol = 1.13 * (784 + 2) * 2.0 ** -23 * (d.abs() @ v.abs().t() + bias.abs())
            tol += 3.3e-7 * linear.abs().clamp_min(1) + 2.0 ** -23 * linear.abs()
            assert ((a - b).abs() <= 2 * tol).all()
        else:
            assert (a - b).norm() <= 2 * (2.0 ** -8 * b.norm() + 1.13 * 2.0 ** -13 * linear.norm())

    alone = [cr.fp8_linear(p, w, out_dtype=out, gelu=True) for w in ws]
    wide = torch.full((m, 520), 5.0, dtype=out, device="cuda")
    outs = [wide[:, 3:303], wide[:, 310:387], wide[:, 388:388], wide[:, 389:517]]
    got = cr.fp8_linear_grouped(p, ws, outs, out_dtype=out, gelu=True)
    for a, b, w in zip(got, alone, ws):
        check(a, b, w)
    for a, b in ((0, 3), (303, 310), (387, 389), (517, 520)):
        assert (wide[:, a:b] == 5.0).all()
    # an unpacked activation gives the same
    for a, b, w in zip(cr.fp8_linear_grouped(x, ws, out_dtype=out, gelu=True), alone, ws):
        check(a, b, w)


def test_empty_calls():
    w = cr.fp8_quantize_weights(torch.randn(64, 256).cuda())
    assert cr.fp8_linear(torch.empty(0, 256, device="cuda"), w).shape == (0, 64)
    none = cr.fp8_quantize_weights(torch.empty(0, 256, device="cuda"))
    assert cr.fp8_linear(torch.randn(5, 256, device="cuda"), none).shape == (5, 0)


def test_results_do_not_vary():
    """The same call twice gives the same bits (no sum depends on timing)."""
    for m in (1, 16, 50, 333):
        x = _inputs(m, 4112, torch.bfloat16, m).cuda()
        w = cr.fp8_quantize_weights(torch.randn(640, 4112).cuda())
        first = cr.fp8_linear(x, w)
        for _ in range(5):
            assert torch.equal(cr.fp8_linear(x, w), first)


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("m", [3, 70, 300])
def test_scales_at_the_ends_of_their_range(m, out):
    """Scale bytes from 0 (2^-127) to 254 (2^127) in both operands, each value finite in float32 (7/8 of
    2^127 at most; 7 times it would not be) and the products within its normal range: exact."""
    n, k = 640, 128
    g = torch.Generator().manual_seed(m)
    qx = torch.randint(1, 8, (m, k), generator=g).float() / 8
    qw = torch.randint(1, 8, (n, k), generator=g).float() / 8
    for pair in ((0, 240), (1, 239), (3, 254), (127, 60), (240, 0), (254, 3), (239, 1)):
        sx = torch.full((1, (m + 3) // 4 * 4), pair[0], dtype=torch.uint8).view(E8M0).cuda().t()[:m]
        sw = torch.full((5, 1), pair[1], dtype=torch.uint8).view(E8M0).cuda()
        y = cr.fp8_linear(cr.Fp8Activation(qx.to(E4M3).cuda(), sx), cr.Fp8Weights(qw.to(E4M3).cuda(), sw),
                          out_dtype=out)
        want = (qx.double() @ qw.double().t()) * 2.0 ** (sum(pair) - 254)
        assert torch.equal(y.cpu(), want.float().to(out)), pair


def _on_gpu(d, w):
    """d W^T in float64 (large references)."""
    return (d.cuda() @ w.cuda().t()).cpu()


WIDE = [(4096, 4096, 384), (4099, 4200, 400), (8200, 2050, 1040), (300, 33000, 656), (33000, 250, 528),
        (4096, 4096, 2064), (2500, 4000, 400), (1700, 3900, 656), (520, 17000, 656), (129, 66000, 528)]


@pytest.mark.parametrize("f32", [False, True], ids=["e8m0", "f32scale"])
@pytest.mark.parametrize("m,n,k", WIDE)
def test_large_outputs_small_integers(m, n, k, f32):
    """Outputs with large tiles for every CU or most of them, whole and ragged."""
    print(f"[gpu] fp8 linear large integers {m}x{n}x{k} f32scale={f32}", flush=True)
    x, w = _integers(m, n, k, f32, m + n + k)
    want = _on_gpu(ref.dequantised_rows(x.q, x.scale), ref.dequantised_weights(w.q, w.scale))
    want += w.bias.cpu().double()
    y = cr.fp8_linear(x, w, out_dtype=torch.bfloat16)
    assert torch.equal(y.cpu(), want.float().to(torch.bfloat16))
    # rows that allow no wide stores, nothing beside them written
    wide = torch.full((m, n + 3), 7.0, dtype=torch.bfloat16, device="cuda")
    cr.fp8_linear(x, w, out=wide[:, 1:n + 1])
    assert torch.equal(wide[:, 1:n + 1], y)
    assert (wide[:, 0] == 7).all() and (wide[:, n + 1:] == 7).all()


@pytest.mark.parametrize("gelu", [False, True], ids=["", "gelu"])
def test_large_grouped_random(gelu):
    m, k = 4100, 1296
    print(f"[gpu] fp8 grouped large gelu={gelu}", flush=True)
    g = torch.Generator().manual_seed(9)
    x = _inputs(m, k, torch.bfloat16, 3)
    ws = [cr.fp8_quantize_weights((torch.randn(n, k, generator=g) * 0.02).cuda(),
                                  torch.randn(n, generator=g).cuda() if n != 1000 else None)
          for n in (2000, 1000, 1552)]
    d, _ = ref.pack(x)
    for y, w in zip(cr.fp8_linear_grouped(x.cuda(), ws, out_dtype=torch.bfloat16, gelu=gelu), ws):
        linear = _on_gpu(d, ref.dequantised_weights(w.q, w.scale))
        if w.bias is not None:
            linear += w.bias.cpu().double()
        want = ref.gelu(linear) if gelu else linear
        off = (y.cpu().double() - want).norm()
        assert off <= 2.0 ** -8 * want.norm() + (1.13 if gelu else 1.0) * 2.0 ** -13 * linear.norm()


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("m,k", [(1, 16), (1, 49152), (2, 24576), (2, 24592), (9, 5120), (16, 2960), (16, 144),
                                 (3, 13824)])
def test_unpacked_rows_equal_packed_rows(m, k, out):
    """Quantised inside the linear or before it, with more and fewer weight rows than CUs take: the
    same bits where every sum is exact (small integers: below 2^24 in units of 2^-6)."""
    print(f"[gpu] fp8 rows {m}x{k} {out}", flush=True)
    g = torch.Generator().manual_seed(k)
    for dt in (torch.float32, torch.bfloat16):
        wide = torch.randint(-2, 3, (m, 2 * k), generator=g).to(dt).cuda()
        x = wide[:, k:]  # rows 2 k apart
        for n in (50, 8300):
            w = cr.fp8_quantize_weights(torch.randint(-2, 3, (n, k), generator=g).float().cuda() / 8,
                                        torch.randint(-9, 10, (n,), generator=g).float().cuda() / 8)
            p = cr.fp8_pack_activations(x)
            y = cr.fp8_linear(x, w, out_dtype=out)
            assert torch.equal(y, cr.fp8_linear(p, w, out_dtype=out))
            if n == 50:
                want = x.cpu().double() @ ref.dequantised_weights(w.q, w.scale).t() + w.bias.cpu().double()
                assert torch.equal(y.cpu(), want.float().to(out))


@pytest.mark.parametrize("f32", [False, True], ids=["e8m0", "f32scale"])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("m,n", [(1, 100), (33, 4090), (70, 2500), (50, 6000), (130, 5000), (60, 17000), (250, 5100),
                                 (1100, 2000), (2113, 2100)])
def test_every_tile_size(m, n, out, f32):
    """Few rows take small output tiles and many take larger ones, with the blocks of features shared
    among waves or not: exact sums are the same for all, and random ones within the tolerance."""
    print(f"[gpu] fp8 linear tiles of {m}x{n} {out} f32scale={f32}", flush=True)
    for k in (400, 1296):  # 4 and 11 blocks
        x, w = _integers(m, n, k, f32, m + n)
        y = cr.fp8_linear(x, w, out_dtype=out)
        want = _on_gpu(ref.dequantised_rows(x.q, x.scale), ref.dequantised_weights(w.q, w.scale))
        want += w.bias.cpu().double()
        assert torch.equal(y.cpu(), want.float().to(out))

    g = torch.Generator().manual_seed(n)
    k = 1296
    W = cr.fp8_quantize_weights((torch.randn(n, k, generator=g) * 0.02).cuda())
    if f32:
        W.scale = W.scale.float() * 1.3
    x = cr.fp8_pack_activations(_inputs(m, k, torch.bfloat16, m).cuda())
    y = cr.fp8_linear(x, W, out_dtype=out).cpu().double()
    d, w = ref.dequantised_rows(x.q, x.scale), ref.dequantised_weights(W.q, W.scale)
    want = _on_gpu(d, w)
    if out == torch.float32:
        assert ((y - want).abs() <= (k + 2) * 2.0 ** -23 * _on_gpu(d.abs(), w.abs())).all()
    else:
        assert (y - want).norm() <= (2.0 ** -8 + 2.0 ** -13) * want.norm()
