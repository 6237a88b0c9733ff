"""Calls of more work than one launch's grid can name (2^32 - 1 threads along an axis) (GPU).

The header allows up to 2^31 - 1 rows, tokens and weight rows.  Each call here is just past what one
launch of its kernel takes and is compared with the same rows called in parts.
"""

import pytest
import torch

import hadamard_rotated_int8_amd as cr

pytestmark = pytest.mark.gpu

E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


@pytest.fixture(autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    cr.lib()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()  # (tens of GB each)


def test_norm_rows_of_one_wave():
    """64 threads to a row: 2^26 rows are 2^32 threads."""
    m, k = 2 ** 26 + 7, 16
    print(f"[gpu] block_norm {m}x{k}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(m, k, generator=g, device="cuda", dtype=torch.bfloat16)
    scale = torch.randn(3, k, generator=g, device="cuda")
    norm = cr.Norm("layer", 1e-5)
    y = cr.block_norm(x, norm, scale[0])
    half = 2 ** 25 + 1
    for at in (slice(0, half), slice(half, m)):
        assert torch.equal(y[at], cr.block_norm(x[at], norm, scale[0]))
    del y
    # groups: the rows behind the first launch find their own vectors
    m -= m % 3
    y = cr.block_norm(x[:m], norm, scale)
    for i in range(3):
        at = slice(i * (m // 3), (i + 1) * (m // 3))
        assert torch.equal(y[at], cr.block_norm(x[at], norm, scale[i]))


def test_norm_rows_of_several_waves():
    """Rows of 1032 features take 128 threads each: 2^25 rows are 2^32."""
    m, k = 2 ** 25 + 3, 1032
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB")
    print(f"[gpu] block_norm {m}x{k} in place", flush=True)
    x = torch.empty(m, k, device="cuda", dtype=torch.bfloat16)
    g = torch.Generator(device="cuda").manual_seed(2)
    part = torch.randn(2 ** 16, k, generator=g, device="cuda").to(torch.bfloat16)
    for at in range(0, m, 2 ** 16):
        x[at:at + 2 ** 16] = part[:m - at]
    norm = cr.Norm("rms", 1e-5)
    want = cr.block_norm(part, norm)
    cr.block_norm(x, norm, out=x)
    for at in range(0, m, 2 ** 16):
        assert torch.equal(x[at:at + 2 ** 16], want[:m - at]), at


def test_rope_tokens():
    """Sixteen tokens to a workgroup of 256: 2^28 tokens are 2^32 threads."""
    t = 2 ** 28 + 21
    print(f"[gpu] rope {t} tokens", flush=True)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(t, 1, 2, generator=g, device="cuda", dtype=torch.bfloat16)
    p = torch.arange(t, device="cuda", dtype=torch.int32)
    plan = cr.RopePlan(torch.tensor([0.37], dtype=torch.float64, device="cuda"))
    y = cr.rope(x, plan, p)
    half = 2 ** 27 + 3
    for at in (slice(0, half), slice(half, t)):
        assert torch.equal(y[at], cr.rope(x[at], plan, p[at]))


@pytest.mark.parametrize("rows,n", [(True, 2 ** 28 + 40), (False, 2 ** 30 + 70)], ids=["unpacked", "packed"])
def test_linear_weight_rows(rows, n):
    """One row of X through very many weight rows: 512 threads to 32 of them unpacked, 256 to 64 packed."""
    k = 16
    print(f"[gpu] fp8 linear 1x{n}x{k} unpacked={rows}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randint(-3, 4, (1, k), generator=g, device="cuda").float()
    period = 2 ** 20 + 128
    codes = torch.randint(-2, 3, (period, k), generator=g, device="cuda").float().to(E4M3)
    q = torch.empty(n, k, dtype=E4M3, device="cuda")
    for at in range(0, n, period):
        q.view(torch.uint8)[at:at + period] = codes.view(torch.uint8)[:n - at]
    scale = torch.full((-(-n // 128), 1), 127, dtype=torch.uint8, device="cuda").view(E8M0)
    w = cr.Fp8Weights(q, scale)
    y = cr.fp8_linear(x if rows else cr.fp8_pack_activations(x), w, out_dtype=torch.bfloat16)
    want = (x.double() @ codes.float().double().t().contiguous()).to(torch.bfloat16)
    for at in range(0, n, period):
        assert torch.equal(y[:, at:at + period], want[:, :n - at]), at


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows", [True, False], ids=["unpacked", "packed"])
def test_linear_of_the_most_weight_rows(rows, out):
    """2^31 - 1 weight rows, outputs with room for a vector store behind the last one: what lies there
    stays (a column number plus 4 does not fit 32 bits)."""
    n, k = 2 ** 31 - 1, 16
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB")
    print(f"[gpu] fp8 linear 2x{n}x{k} {out} unpacked={rows}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randint(-3, 4, (2, k), generator=g, device="cuda").float()
    period = 2 ** 24
    codes = torch.randint(-2, 3, (period, k), generator=g, device="cuda").float().to(E4M3)
    q = torch.empty(n, k, dtype=E4M3, device="cuda")
    for at in range(0, n, period):
        q.view(torch.uint8)[at:at + period] = codes.view(torch.uint8)[:n - at]
    scale = torch.full((-(-n // 128), 1), 127, dtype=torch.uint8, device="cuda").view(E8M0)
    y = torch.full((2, n + 1), 9.0, dtype=out, device="cuda")
    cr.fp8_linear(x if rows else cr.fp8_pack_activations(x), cr.Fp8Weights(q, scale), out=y[:, :n])
    want = (x.double() @ codes.float().double().t().contiguous()).to(out)
    for at in range(0, n, period):
        assert torch.equal(y[:, at:min(at + period, n)], want[:, :n - at]), at
    assert (y[:, n] == 9).all()
