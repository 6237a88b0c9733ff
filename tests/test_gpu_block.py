"""A transformer block's operators run together, as a model uses them (GPU).

Every stage is compared with the 64-bit reference of that stage on the values
the stage really got, with the tolerances that the modules of the single
operators derive (an FP8 code that falls to the other side of a tie would
make errors of a whole block incomparable).  Captured graphs, side streams
and repeated calls have to give the eager call's bits.
"""

import pytest
import torch

import block_reference as ref
import hadamard_rotated_int8_amd as cr
import test_gpu_block_norm as norms
import test_gpu_rope as ropes

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HEADS, D, K, HIDDEN = 5, 128, 640, 1296


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    cr.lib()
    yield
    torch.cuda.synchronize()


class Block:
    """Weights of one block; ``run`` returns everything it computed."""

    def __init__(self, batch, seed=0, f32_scale=False):
        g = torch.Generator().manual_seed(seed)

        def weights(n, k):
            w = cr.fp8_quantize_weights((torch.randn(n, k, generator=g) * k ** -0.5).cuda(),
                                        (torch.randn(n, generator=g) * 0.1).cuda())
            if f32_scale:
                w.scale = w.scale.float() * 0.9
            return w

        self.qkv = [weights(K, K) for _ in range(3)]
        self.o, self.up, self.down = weights(K, K), weights(HIDDEN, K), weights(K, HIDDEN)
        self.mod = (torch.randn(batch, 6 * K, generator=g) * 0.3).cuda()  # as a projection writes it
        self.post = cr.Norm("rms", 1e-6, (torch.rand(K, generator=g) + 0.5).cuda())
        self.norm = cr.Norm("layer", 1e-6)
        self.plan = cr.rope_plan(D, axes=(44, 42, 42))

    def part(self, i):
        return self.mod[:, i * K:(i + 1) * K]

    def run(self, x, positions, batch):
        m = x.shape[0]
        heads = (batch, m // batch, HEADS, D)
        s = {}
        s["p"] = cr.block_norm(x, self.norm, self.part(0), self.part(1), pack=True)
        s["qkv"] = cr.fp8_linear_grouped(s["p"], self.qkv, out_dtype=torch.bfloat16)
        s["turned"] = cr.rope([t.view(heads) for t in s["qkv"][:2]], self.plan, positions)
        # (stands for the attention: something that every one of the three goes into)
        s["a"] = (s["turned"][0] * s["turned"][1]).view(m, K) + s["qkv"][2]
        s["o"] = cr.fp8_linear(s["a"], self.o)
        s["h"], s["p2"] = cr.block_update(x, s["o"], self.part(2), post=self.post, norm=self.norm,
                                          scale=self.part(3), shift=self.part(4), pack=True)
        s["up"] = cr.fp8_linear(s["p2"], self.up, out_dtype=torch.bfloat16, gelu=True)
        s["down"] = cr.fp8_linear(s["up"], self.down)
        s["h2"], s["y"] = cr.block_update(s["h"], s["down"], self.part(5), norm=self.norm)
        return s


def _flat(s):
    for v in s.values():
        for t in v if isinstance(v, list) else [v]:
            if isinstance(t, cr.Fp8Activation):
                yield t.q.view(torch.uint8)
                yield t.scale.view(torch.uint8)
            else:
                yield t


def _inputs(batch, tokens, seed=1):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(batch * tokens, K, generator=g).to(torch.bfloat16)
    return x, torch.randint(0, 200, (tokens, 3), generator=g, dtype=torch.int32)


def _check_linear(y, rows, w, gelu=False):
    weights = ref.dequantised_weights(w.q, w.scale)
    linear = rows @ weights.t() + w.bias.cpu().double()
    want = ref.gelu(linear) if gelu else linear
    off = (y.cpu().double() - want).abs()
    if y.dtype == torch.float32:
        size = rows.abs() @ weights.abs().t() + w.bias.cpu().double().abs()
        assert (off <= (rows.shape[1] + 2) * 2.0 ** -23 * size).all()
    else:
        assert off.norm() <= 2.0 ** -8 * want.norm() + 1.13 * 2.0 ** -13 * linear.norm()


@pytest.mark.parametrize("f32_scale", [False, True], ids=["e8m0", "f32scale"])
@pytest.mark.parametrize("batch,tokens", [(1, 1), (2, 7), (2, 45), (1, 333)])
def test_block(batch, tokens, f32_scale):
    print(f"[gpu] block {batch}x{tokens} f32scale={f32_scale}", flush=True)
    b = Block(batch, f32_scale=f32_scale)
    x, positions = _inputs(batch, tokens)
    s = b.run(x.cuda(), positions.cuda(), batch)
    m = batch * tokens

    y = cr.block_norm(x.cuda(), b.norm, b.part(0), b.part(1), out_dtype=torch.float32).cpu()
    packed, byte = ref.pack(y)
    rows = ref.dequantised_rows(s["p"].q, s["p"].scale)
    assert torch.equal(rows, packed)
    for t, w in zip(s["qkv"], b.qkv):
        _check_linear(t, rows, w)
    for t, before in zip(s["turned"], s["qkv"]):
        ropes._check(t, before.cpu().view(batch, tokens, HEADS, D), b.plan, positions)
    rows, _ = ref.pack(s["a"].cpu())
    _check_linear(s["o"], rows, b.o)

    def check_update(h, x, branch, gate, post, pre=(), y=None, scale=None, shift=None):
        want_h, want_y = ref.block(x.cpu(), branch.cpu(), gate, 1.0, post, pre or None, scale, shift)
        normed = branch.cpu().double() if post is None else ref.norm(branch.cpu(), *post)
        parts = x.cpu().double().abs() + ref.rows_of(gate, m).abs() * normed.abs()
        grown = parts.norm(dim=1) / want_h.norm(dim=1)
        rel = ((128 * (1 + norms._spread(branch.cpu(), "rms")) if post else 0 * grown) + 8) * U * grown
        norms._check(h, want_h, torch.bfloat16, rel)
        if y is not None:
            parts = want_y.abs() if scale is None else \
                ref.norm(want_h, *pre).abs() * (1 + ref.rows_of(scale, m)).abs() + \
                ref.rows_of(shift, m).abs()
            a = 1 + norms._spread(want_h, "layer")
            norms._check(y, want_y, y.dtype,
                         (2 * rel * a + (128 * a + 8) * U) * 4 * parts.norm(dim=1) / want_y.norm(dim=1))

    post = ("rms", 1e-6, b.post.weight)
    h, y = cr.block_update(x.cuda(), s["o"], b.part(2), post=b.post, norm=b.norm, scale=b.part(3),
                           shift=b.part(4), out_dtype=torch.float32)
    check_update(s["h"], x, s["o"], b.part(2), post, ("layer", 1e-6), y, b.part(3), b.part(4))
    assert torch.equal(h, s["h"])
    rows, _ = ref.pack(y.cpu())
    assert torch.equal(rows, ref.dequantised_rows(s["p2"].q, s["p2"].scale))
    _check_linear(s["up"], rows, b.up, gelu=True)
    rows, _ = ref.pack(s["up"].cpu())
    _check_linear(s["down"], rows, b.down)
    check_update(s["h2"], s["h"], s["down"], b.part(5), None, ("layer", 1e-6), s["y"])


@pytest.mark.parametrize("batch,tokens", [(1, 1), (2, 20), (1, 130)])
def test_captured_block_replays(batch, tokens):
    """A block in a graph, replayed on new inputs with eager work of the same operators between the
    replays: the eager bits each time."""
    print(f"[gpu] block graph {batch}x{tokens}", flush=True)
    b = Block(batch)
    x, positions = (t.cuda() for t in _inputs(batch, tokens))
    b.run(x, positions, batch)  # (loads the library before the capture)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s = b.run(x, positions, batch)
    for i in range(4):
        new, at = _inputs(batch, tokens, 10 + i)
        x.copy_(new)
        positions.copy_(at)
        graph.replay()
        got = [t.clone() for t in _flat(s)]
        want = b.run(new.cuda(), at.cuda(), batch)
        torch.cuda.synchronize()
        for g, w in zip(got, _flat(want)):
            assert torch.equal(g, w)


def test_two_graphs_and_two_streams():
    """Two captured blocks that share their weights replay side by side on two streams (no memory of
    a call is shared with another's)."""
    b = Block(1)
    runs = []
    for i in range(2):
        x, positions = (t.cuda() for t in _inputs(1, 70, 20 + i))
        want = [t.clone() for t in _flat(b.run(x, positions, 1))]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s = b.run(x, positions, 1)
        runs.append((graph, s, want, torch.cuda.Stream(), x, positions))
    for _ in range(3):
        for graph, _, _, stream, _, _ in runs:
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                graph.replay()
        for run in runs:
            torch.cuda.current_stream().wait_stream(run[3])
        for _, s, want, *_ in runs:
            for g, w in zip(_flat(s), want):
                assert torch.equal(g, w)


def test_calls_go_to_the_current_stream():
    """Work queued before the call on the current stream is seen by it: the inputs are filled there."""
    b = Block(1)
    x, positions = (t.cuda() for t in _inputs(1, 50))
    want = [t.clone() for t in _flat(b.run(x, positions, 1))]
    for _ in range(3):
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            late = torch.zeros_like(x)
            big = torch.zeros(1 << 26, device="cuda")  # something to wait for
            for _ in range(8):
                big.add_(1)
            late.copy_(x)
            got = b.run(late, positions, 1)
        stream.synchronize()
        for g, w in zip(_flat(got), want):
            assert torch.equal(g, w)


def test_beside_the_int8_linears():
    """block_norm feeds the INT8 linears and their float32 outputs come back through block_update;
    the FP8 linears see the same rows to within both quantisations."""
    g = torch.Generator().manual_seed(5)
    m, k = 60, 1024
    x = torch.randn(m, k, generator=g).to(torch.bfloat16).cuda()
    w = (torch.randn(k, k, generator=g) * k ** -0.5).cuda()
    y = cr.block_norm(x, cr.Norm("rms"))
    exact = y.double().cpu() @ w.double().cpu().t()
    int8 = cr.linear(cr.pack_activations(y.float(), 256), cr.quantize_weights(w, 256))
    fp8 = cr.fp8_linear(y, cr.fp8_quantize_weights(w))
    # a step of 2^-3 relative at most: 2^-4 per code, both operands, independent over 1024 features
    assert (fp8.cpu().double() - exact).norm() <= 2.0 ** -4 * exact.norm()
    assert (int8.cpu().double() - exact).norm() <= 2.0 ** -4 * exact.norm()
    for branch in (int8, fp8):
        h, none = cr.block_update(x, branch, residual_scale=0.5)
        assert none is None
        want = (0.5 * x.double() + branch.double()).cpu()
        # one fused or two roundings in float32, one to bfloat16
        tol = 2.0 ** -8 * want.abs() + 4 * U * (x.double().abs() + branch.double().abs()).cpu()
        assert ((h.cpu().double() - want).abs() <= tol).all()


def _refused(fn, *args, **kw):
    with pytest.raises((ValueError, cr.ConvrotError)):
        fn(*args, **kw)


def test_linear_refusals():
    w = cr.fp8_quantize_weights(torch.randn(64, 256, device="cuda"), torch.randn(64, device="cuda"))
    x = torch.randn(20, 256, device="cuda")
    p = cr.fp8_pack_activations(x)
    _refused(cr.fp8_linear, x.half(), w)
    _refused(cr.fp8_linear, x.t(), w)
    _refused(cr.fp8_linear, x[:, :128], w)  # another K
    _refused(cr.fp8_linear, x[:, :250], w)  # K no multiple of 16
    _refused(cr.fp8_linear, cr.fp8_pack_activations(x[:, :128]), w)
    _refused(cr.fp8_linear, x, w, out_dtype=torch.float16)
    _refused(cr.fp8_linear, x, w, out=torch.empty(20, 65, device="cuda"))
    _refused(cr.fp8_linear, x, w, out=torch.empty(20, 64, device="cuda", dtype=torch.float16))
    _refused(cr.fp8_linear, x, w, out=torch.empty(64, 20, device="cuda").t())
    _refused(cr.fp8_linear, x, w, out=torch.empty(64, device="cuda").expand(20, 64))
    _refused(cr.fp8_linear, x, w, out=torch.empty(20, 64))
    _refused(cr.fp8_linear_grouped, x, [])
    _refused(cr.fp8_linear_grouped, x, [w] * (cr.MAX_GROUPED + 1))
    y = torch.empty(20, 64, device="cuda")
    _refused(cr.fp8_linear_grouped, x, [w, w], [y])
    _refused(cr.fp8_linear_grouped, x, [w, w], [y, y])
    _refused(cr.fp8_linear, x, cr.Fp8Weights(w.q, w.scale[:, :1], None))
    _refused(cr.fp8_linear, x, cr.Fp8Weights(w.q, w.scale.view(torch.uint8), None))
    _refused(cr.fp8_linear, x, cr.Fp8Weights(w.q.view(torch.uint8), w.scale, None))
    _refused(cr.fp8_linear, x, cr.Fp8Weights(w.q, w.scale, w.bias.double()))
    _refused(cr.fp8_linear, x, cr.Fp8Weights(w.q, w.scale, w.bias[:3]))
    _refused(cr.fp8_linear, x, cr.Fp8Weights(w.q.cpu(), w.scale, None))
    _refused(cr.fp8_linear, cr.Fp8Activation(p.q[:, :128], p.scale), w)
    _refused(cr.fp8_linear, cr.Fp8Activation(p.q, p.scale.contiguous()), w)
    _refused(cr.fp8_linear, cr.Fp8Activation(p.q[:19], p.scale[:19].t().contiguous().t()), w)  # no padding
    _refused(cr.fp8_pack_activations, x[:, :250])
    _refused(cr.fp8_pack_activations, x, cr.fp8_pack_activations(x[:10]))
    _refused(cr.fp8_quantize_weights, x.half())
    _refused(cr.fp8_quantize_weights, x[:, :250].contiguous())


def test_norm_refusals():
    x = torch.randn(20, 256, device="cuda")
    n = cr.Norm("rms")
    _refused(cr.block_norm, x.half(), n)
    _refused(cr.block_norm, x[0], n)
    _refused(cr.block_norm, x, cr.Norm("batch"))
    _refused(cr.block_norm, x, cr.Norm("rms", -1.0))
    _refused(cr.block_norm, x, cr.Norm("rms", 1e-6, torch.ones(255, device="cuda")))
    _refused(cr.block_norm, x, cr.Norm("rms", 1e-6, torch.ones(256)))
    _refused(cr.block_norm, x, n, torch.ones(3, 256, device="cuda"))  # 3 does not divide 20
    _refused(cr.block_norm, x, n, torch.ones(256, device="cuda", dtype=torch.float16))
    _refused(cr.block_norm, x, n, out_dtype=torch.float16)
    _refused(cr.block_norm, x, n, out=torch.empty(20, 255, device="cuda"))
    _refused(cr.block_norm, x, n, out=x, out_dtype=torch.bfloat16)
    _refused(cr.block_norm, x[:, :250], n, pack=True)
    _refused(cr.block_norm, x, n, out=x, pack=True)
    _refused(cr.block_norm, torch.empty(1, cr.MAX_NORM_K + 1, device="cuda"), n)
    _refused(cr.block_update, x, x[:10])
    _refused(cr.block_update, x, x.half())
    _refused(cr.block_update, x, x, gate=torch.ones(256))
    _refused(cr.block_update, x, x, out_h=x.bfloat16())
    _refused(cr.block_update, x, x, pack=True)  # nothing to pack
    _refused(cr.block_update, x, x, out=x)
    _refused(cr.block_update, x, x.clone(), norm=n, out_h=x, out=x)  # both over x
    _refused(cr.block_update, x, x.clone(), norm=n, out_h=x, out=x[:, :])
    _refused(cr.block_norm, x.bfloat16().view(-1)[:2560].view(10, 256), n, out=None, out_dtype=torch.int8)


def test_rope_refusals():
    x = torch.randn(20, 4, 64, device="cuda")
    plan = cr.rope_plan(64)
    at = torch.arange(20, device="cuda")
    _refused(cr.rope, x.half(), plan, at)
    _refused(cr.rope, x[0], plan, at)
    _refused(cr.rope, x, plan, at[:19])
    _refused(cr.rope, x, plan, at.cpu())
    _refused(cr.rope, x, plan, at.to(torch.int16))
    _refused(cr.rope, x[..., :32], plan, at)  # the slice ends outside the head
    _refused(cr.rope, x, cr.rope_plan(32, start=33), at)
    _refused(cr.rope, [x] * (cr.MAX_ROPE_TENSORS + 1), plan, at)
    _refused(cr.rope, [x, x[:10]], plan, at)
    _refused(cr.rope, [x, x], plan, at, out=[x, x])  # it would turn twice, or once
    _refused(cr.rope, x, plan, at, out=torch.empty(20, 4, 63, device="cuda"))
    _refused(cr.rope, x, plan, at, out=torch.empty(20, 1, 64, device="cuda").expand(20, 4, 64))
    _refused(cr.rope, x, cr.rope_plan(64, axes=(32, 32)), at)
    _refused(cr.rope, x, cr.RopePlan(plan.inv_freq.float()), at)
    _refused(cr.rope, x, cr.RopePlan(plan.inv_freq, "spiral"), at)
