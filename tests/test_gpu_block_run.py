"""An image model's block as one run of operators: group norm, FP8 linears, norms, rotary positions, the
tokens' attention to one another and to a prompt, and a gated feed-forward with its way back.  Each new
operator's output against the 64-bit reference of what it was given, and the whole run the same bits
captured and replayed, on other streams, and on two streams at once (GPU)."""

import pytest
import torch

import hadamard_rotated_int8_amd as cr
import test_gpu_gated as gated
import test_gpu_group_norm as group_norm
from attention_reference import attention_ref

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


class Block:
    def __init__(self, hidden, heads, inner, states, seed=0):
        g = torch.Generator().manual_seed(seed)

        def weights(n, k):
            w = torch.randn(n, k, generator=g) * k ** -0.5
            return cr.fp8_quantize_weights(w.cuda(), (0.1 * torch.randn(n, generator=g)).cuda())

        self.heads, self.d = heads, hidden // heads
        self.groups, self.affine = 8, group_norm._affine(64, torch.float32)
        self.enter = weights(hidden, 64)
        self.qkv = [weights(hidden, hidden) for _ in range(3)]
        self.out, self.query, self.out2 = (weights(hidden, hidden) for _ in range(3))
        self.key_value = weights(2 * hidden, states)
        self.gate, self.up, self.down = weights(inner, hidden), weights(inner, hidden), weights(hidden, inner)
        self.back = cr.fp8_transpose_weights([self.gate, self.up])
        self.plan = cr.rope_plan(self.d, axes=(self.d // 2, self.d // 2))
        self.scale = (0.1 * torch.randn(hidden, generator=g)).cuda()

    def __call__(self, image, prompt, lengths, dy):
        r = {}
        batch, height, width, _ = image.shape
        tokens, heads, d = height * width, self.heads, self.d
        norm = cr.Norm("layer")
        at = torch.arange(tokens, dtype=torch.int32, device="cuda")
        positions = torch.stack([at // width, at % width], dim=1)
        r["image"] = cr.group_norm(image, self.groups, *self.affine, silu=True, out_dtype=BF16)
        h = cr.fp8_linear(r["image"].view(batch * tokens, -1), self.enter, out_dtype=BF16)
        p = cr.block_norm(h, norm, self.scale, pack=True)
        q, k, v = (t.view(batch, tokens, heads, d) for t in cr.fp8_linear_grouped(p, self.qkv, out_dtype=BF16))
        q, k = cr.rope([q, k], self.plan, positions.expand(batch, tokens, 2).contiguous())
        r["self"] = (q, k, v, cr.attention(q, k, v))
        a = r["self"][3].view(batch * tokens, -1)
        h, p = cr.block_update(h, cr.fp8_linear(a, self.out, out_dtype=BF16), norm=norm, scale=self.scale, pack=True)
        q = cr.fp8_linear(p, self.query, out_dtype=BF16).view(batch, tokens, heads, d)
        kv = cr.fp8_linear(prompt.flatten(0, 1), self.key_value, out_dtype=BF16).view(batch, -1, 2 * heads, d)
        k, v = kv[:, :, :heads], kv[:, :, heads:]
        r["cross"] = (q, k, v, cr.attention(q, k, v, lengths=lengths))
        a = r["cross"][3].view(batch * tokens, -1)
        h, p = cr.block_update(h, cr.fp8_linear(a, self.out2, out_dtype=BF16), norm=norm, scale=self.scale, pack=True)
        r["packed"] = p
        r["y"], r["kept"] = cr.fp8_gated(p, self.gate, self.up, out_dtype=BF16, keep=True)
        r["h"], _ = cr.block_update(h, cr.fp8_linear(r["y"], self.down, out_dtype=BF16))
        r["dx"], r["grads"] = cr.fp8_gated_backward(dy, r["kept"], self.back)
        return r


def _tensors(r):
    return [r["image"], r["self"][3], r["cross"][3], r["y"], *r["kept"], r["h"], r["dx"], *r["grads"]]


def _inputs(batch, height, width, states, length, inner, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(BF16)

    lengths = torch.randint(0, length + 1, (batch,), generator=g, device="cuda", dtype=torch.int32)
    return [normal(batch, height, width, 64), normal(batch, length, states), lengths,
            normal(batch * height * width, inner)]


SHAPES = pytest.mark.parametrize("batch, height, width, hidden, heads, length, inner", [
    (1, 1, 1, 128, 2, 1, 144), (2, 9, 12, 256, 4, 20, 400), (3, 33, 31, 512, 4, 77, 1040)])


@SHAPES
def test_each_against_its_reference(batch, height, width, hidden, heads, length, inner):
    block = Block(hidden, heads, inner, 96)
    image, prompt, lengths, dy = _inputs(batch, height, width, 96, length, inner, 1)
    r = block(image, prompt, lengths, dy)
    ref, tol = group_norm._reference(image, 8, *block.affine, 1e-6, True, BF16)
    assert ((r["image"].double() - ref).abs() <= tol).all()
    for name, kw in (("self", {}), ("cross", {"lengths": lengths})):
        q, k, v, out = r[name]
        ref, tol = attention_ref(q, k, v, **kw)
        assert ((out.cpu().double() - ref).abs() <= tol).all()
    gated._check(r["packed"], block.gate, block.up, "silu", BF16, r["y"], r["kept"])
    assert all(not t.isnan().any() for t in _tensors(r))


@SHAPES
def test_the_same_bits_captured_and_on_other_streams(batch, height, width, hidden, heads, length, inner):
    block = Block(hidden, heads, inner, 96)
    sets = [_inputs(batch, height, width, 96, length, inner, seed) for seed in range(3)]
    want = [_tensors(block(*s)) for s in sets]
    static = [t.clone() for t in sets[0]]
    block(*static)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _tensors(block(*static))
    for s, w in zip(sets + sets[:1], want + want[:1]):
        for t, v in zip(static, s):
            t.copy_(v)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, w))
        block(*sets[1])  # (other work between the replays)
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    results = [None, None]
    for _ in range(2):
        for i, stream in enumerate(streams):
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                results[i] = _tensors(block(*sets[i]))
    torch.cuda.synchronize()
    for r, w in zip(results, want):
        assert all(torch.equal(a, b) for a, b in zip(r, w))
