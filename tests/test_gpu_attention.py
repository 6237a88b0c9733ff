"""Attention against its definition in 64 bits: head dimensions, grouped heads, lengths from nothing to
long, hidden keys, strides, splits of the keys, captured calls and other streams."""

import math

import pytest
import torch

import hadamard_rotated_int8_amd as cr
from attention_reference import attention_ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _inputs(batch, m, l, heads, kv, d, seed=0, scale_q=1.5):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rows = torch.randn(batch, l, 2 * kv, d, generator=g, device=DEV).to(torch.bfloat16)
    q = (scale_q * torch.randn(batch, m, heads, d, generator=g, device=DEV)).to(torch.bfloat16)
    return q, rows[:, :, :kv], rows[:, :, kv:]


def _check(q, k, v, out, **kw):
    ref, tol = attention_ref(q, k, v, **kw)
    assert out.dtype == torch.bfloat16 and out.shape == q.shape
    off = (out.cpu().double() - ref).abs()
    worst = (off - tol).max().item()
    assert not out.isnan().any() and worst <= 0, (worst, off.max().item())


@pytest.mark.parametrize("d", [8, 16, 40, 64, 72, 80, 96, 104, 128, 136, 160, 168, 192])
@pytest.mark.parametrize("m, l", [(1, 1), (33, 65), (130, 129)])
def test_head_dimensions(d, m, l):
    q, k, v = _inputs(2, m, l, 2, 2, d, seed=d)
    _check(q, k, v, cr.attention(q, k, v))


@pytest.mark.parametrize("m", [1, 2, 31, 32, 33, 64, 127, 128, 129, 255, 257, 513])
@pytest.mark.parametrize("l", [1, 31, 32, 33, 63, 64, 65, 127, 128, 200])
def test_lengths(m, l):
    q, k, v = _inputs(1, m, l, 1, 1, 64, seed=m * 1000 + l)
    _check(q, k, v, cr.attention(q, k, v))


@pytest.mark.parametrize("heads, kv", [(1, 1), (4, 1), (8, 2), (5, 5), (10, 2), (7, 1), (96, 4)])
@pytest.mark.parametrize("m", [1, 3, 70])
def test_grouped_heads(heads, kv, m):
    q, k, v = _inputs(2, m, 100, heads, kv, 64, seed=heads)
    _check(q, k, v, cr.attention(q, k, v))


@pytest.mark.parametrize("m, l", [(1, 4096), (1, 32760), (5, 10001), (40, 2050), (200, 3001)])
@pytest.mark.parametrize("d", [64, 128, 160])
def test_few_queries_over_many_keys(m, l, d):
    q, k, v = _inputs(1, m, l, 2, 1, d, seed=l)
    _check(q, k, v, cr.attention(q, k, v))


@pytest.mark.parametrize("d, heads, kv, m", [(64, 26, 13, 2555), (128, 24, 24, 2700), (160, 13, 13, 2555)])
def test_a_last_round_of_few_tiles(d, heads, kv, m):
    # (520, 528 or 260 tiles, on 512 places or 256: the keys of the last ones are split)
    l = 1100
    q, k, v = _inputs(1, m, l, heads, kv, d, seed=d)
    mask = torch.rand(1, l, device=DEV, generator=torch.Generator(device=DEV).manual_seed(d)) < 0.5
    mask[0, 500:800] = False
    at = [0, heads // 2, heads - 1]
    for kw in ({}, {"lengths": torch.tensor([1027], dtype=torch.int32, device=DEV)}, {"mask": mask},
               {"lengths": torch.tensor([0], dtype=torch.int32, device=DEV)}):
        out = cr.attention(q, k, v, **kw)
        key = [h // (heads // kv) for h in at]
        _check(q[:, :, at], k[:, :, key], v[:, :, key], out[:, :, at], **kw)


@pytest.mark.parametrize("m", [1, 40, 300])
@pytest.mark.parametrize("l", [77, 300, 5000])
def test_lengths_of_a_batch(m, l):
    q, k, v = _inputs(6, m, l, 2, 2, 64, seed=l)
    lengths = torch.tensor([l, 0, 1, l - 1, l + 5, -3], dtype=torch.int32, device=DEV)
    out = cr.attention(q, k, v, lengths=lengths)
    _check(q, k, v, out, lengths=lengths.clamp(0, l))
    assert (out[1] == 0).all() and (out[5] == 0).all()


@pytest.mark.parametrize("m", [1, 40, 300])
@pytest.mark.parametrize("l", [77, 300, 5000])
def test_masks(m, l):
    q, k, v = _inputs(4, m, l, 2, 1, 128, seed=l)
    g = torch.Generator(device=DEV).manual_seed(l)
    mask = torch.rand(4, l, generator=g, device=DEV) < 0.5
    mask[1] = False
    mask[2] = False
    mask[2, l - 1] = True
    mask[3, :70] = False
    _check(q, k, v, cr.attention(q, k, v, mask=mask), mask=mask)
    lengths = torch.tensor([l, l, l - 1, 72], dtype=torch.int32, device=DEV)
    out = cr.attention(q, k, v, mask=mask, lengths=lengths)
    _check(q, k, v, out, mask=mask, lengths=lengths)
    assert (out[1] == 0).all() and (out[2] == 0).all()
    _check(q, k, v, cr.attention(q, k, v, mask=mask[0]), mask=mask[:1].expand(4, l))


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf, torch.finfo(torch.bfloat16).min])
@pytest.mark.parametrize("m, l", [(1, 300), (70, 300), (300, 77), (2, 5000)])
def test_hidden_keys_hold_anything(bad, m, l):
    q, k, v = _inputs(2, m, l, 2, 2, 64, seed=l)
    k, v = k.clone(), v.clone()
    g = torch.Generator(device=DEV).manual_seed(l)
    mask = torch.rand(2, l, generator=g, device=DEV) < 0.7
    lengths = torch.tensor([l - 3, l // 2], dtype=torch.int32, device=DEV)
    clean = cr.attention(q, k, v, mask=mask, lengths=lengths)
    hidden = ~mask | (torch.arange(l, device=DEV) >= lengths[:, None])
    k[hidden], v[hidden] = bad, bad
    assert torch.equal(cr.attention(q, k, v, mask=mask, lengths=lengths), clean)


def test_a_seen_nan_reaches_its_head_only():
    q, k, v = _inputs(2, 40, 100, 2, 2, 64)
    k = k.clone()
    k[1, 99, 1, 3] = math.nan
    out = cr.attention(q, k, v)
    assert out[1, :, 1].isnan().all()
    assert not out[0].isnan().any() and not out[1, :, 0].isnan().any()
    q = q.clone()
    q[0, 7, 0, 0] = math.nan
    out = cr.attention(q, k, v)
    assert out[0, 7, 0].isnan().all() and not out[0, :7].isnan().any() and not out[0, 8:].isnan().any()


@pytest.mark.parametrize("m, l", [(1, 2000), (64, 500), (300, 500)])
def test_scores_far_apart_and_rising(m, l):
    # scores of hundreds, the largest last, first or all alike: the running maximum moves or stays
    q, k, v = _inputs(1, m, l, 2, 2, 64, seed=7, scale_q=8.0)
    k = k.clone()
    k *= torch.linspace(0.1, 6, l, device=DEV)[None, :, None, None].to(torch.bfloat16)
    _check(q, k, v, cr.attention(q, k, v))
    _check(q, k.flip(1), v, cr.attention(q, k.flip(1), v))
    k[:] = k[:, :1].clone()
    _check(q, k, v, cr.attention(q, k, v))
    ones = torch.ones_like(q)
    lift = (torch.arange(l, device=DEV).float() * 0.37)[None, :, None, None].expand(k.shape).to(torch.bfloat16)
    _check(ones, lift, v, cr.attention(ones, lift, v))
    _check(ones, -lift, v, cr.attention(ones, -lift, v))


@pytest.mark.parametrize("scale", [1e-6, 0.03, 1.0])
def test_scales(scale):
    q, k, v = _inputs(1, 50, 200, 2, 2, 96, seed=3)
    _check(q, k, v, cr.attention(q, k, v, scale=scale), scale=scale)


def test_strides_and_outputs():
    batch, m, l, heads, kv, d = 2, 70, 130, 4, 2, 80
    g = torch.Generator(device=DEV).manual_seed(1)
    rows = torch.randn(batch, m, heads * d + 8, generator=g, device=DEV).to(torch.bfloat16)
    q = rows[:, :, 8:].unflatten(-1, (heads, d))
    head_first = torch.randn(batch, kv, l, 2 * d, generator=g, device=DEV).to(torch.bfloat16)
    k, v = head_first[..., :d].transpose(1, 2), head_first[..., d:].transpose(1, 2)
    ref = cr.attention(q.contiguous(), k.contiguous(), v.contiguous())
    _check(q, k, v, ref)
    assert torch.equal(cr.attention(q, k, v), ref)
    wide = torch.full((batch, heads, m + 3, d + 16), 7.0, dtype=torch.bfloat16, device=DEV)
    out = wide[:, :, 1:m + 1, 8:8 + d].transpose(1, 2)
    assert cr.attention(q, k, v, out=out) is out
    assert torch.equal(out, ref)
    out.fill_(7.0)
    assert (wide == 7.0).all()  # nothing beside it was written
    # one prompt for the whole batch, and no batch at all
    shared = cr.attention(q, k[:1].expand(batch, -1, -1, -1), v[:1].expand(batch, -1, -1, -1))
    assert torch.equal(shared[1], cr.attention(q[1], k[0], v[0]))
    assert torch.equal(shared[0], ref[0])


def test_axes_of_one_may_state_any_stride():
    g = torch.Generator(device=DEV).manual_seed(3)
    flat = torch.randn(3, 4097, generator=g, device=DEV).to(torch.bfloat16)
    q = flat[:1, :64].as_strided((1, 1, 1, 64), (4097, 5, 3, 1))
    k = flat[1].as_strided((1, 32, 1, 64), (9, 128, 1, 1), 4104)
    v = flat[1].as_strided((1, 32, 1, 64), (9, 128, 1, 1), 4104 + 64)
    out = torch.empty(100, dtype=torch.bfloat16, device=DEV).as_strided((1, 1, 1, 64), (3, 1, 7, 1))
    ref = cr.attention(q.contiguous(), k.contiguous(), v.contiguous())
    assert torch.equal(cr.attention(q, k, v), ref)
    assert torch.equal(cr.attention(q, k, v, out=out), ref)


def test_outputs_over_inputs_are_refused():
    q, k, v = _inputs(2, 8, 40, 2, 2, 64)
    space = torch.empty(q.numel() * 2 + 80, dtype=torch.uint8, device=DEV)
    out = space[:q.numel() * 2].view(torch.bfloat16).view(q.shape)
    mask = space[q.numel() * 2 - 16:q.numel() * 2 + 64].view(torch.bool).view(2, 40)
    lengths = space[:8].view(torch.int32)
    for args, kw in (((q, k, v), {"out": q}), ((q, k, v), {"out": out, "mask": mask}),
                     ((q, k, v), {"out": out, "lengths": lengths}), ((out, k, v), {"out": out})):
        with pytest.raises(ValueError, match="over an input"):
            cr.attention(*args, **kw)
    with pytest.raises(ValueError, match="overlap"):
        cr.attention(q, k, v, out=q.new_empty(1, 8, 2, 64).expand(2, 8, 2, 64))


@pytest.mark.parametrize("l", [3, 31, 32, 33, 2049, 4500])
def test_a_mask_at_any_address(l):
    q, k, v = _inputs(2, 130, l, 2, 1, 64, seed=l)
    g = torch.Generator(device=DEV).manual_seed(l)
    wide = torch.rand(2, l + 9, generator=g, device=DEV) < 0.5
    for at in (1, 2, 7):
        _check(q, k, v, cr.attention(q, k, v, mask=wide[:, at:at + l]), mask=wide[:, at:at + l])
    # a byte that is neither 0 nor 1 shows its key too
    odd = (torch.randint(0, 3, (2, l), generator=g, device=DEV, dtype=torch.uint8) * 127)
    _check(q, k, v, cr.attention(q, k, v, mask=odd.view(torch.bool)), mask=odd != 0)


def test_empty_sizes():
    q, k, v = _inputs(2, 5, 7, 2, 2, 64)
    assert (cr.attention(q, k[:, :0], v[:, :0]) == 0).all()
    assert cr.attention(q[:, :0], k, v).shape == (2, 0, 2, 64)
    assert cr.attention(q[:0], k[:0], v[:0]).shape == (0, 5, 2, 64)


@pytest.mark.parametrize("m, l, d", [(1, 5000, 128), (300, 333, 64)])
def test_graphs_and_streams(m, l, d):
    q, k, v = _inputs(2, m, l, 4, 2, d, seed=1)
    lengths = torch.tensor([l, l // 2], dtype=torch.int32, device=DEV)
    want = cr.attention(q, k, v, lengths=lengths)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = cr.attention(q, k, v, lengths=lengths)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    graphs = []
    for _ in range(2):  # (two graphs of one call: each has a workspace of its own)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res = cr.attention(q, k, v, lengths=lengths)
        graphs.append((graph, res))
    for round in range(3):
        q.copy_(_inputs(2, m, l, 4, 2, d, seed=10 + round)[0])
        lengths.fill_(l - round)
        eager = cr.attention(q, k, v, lengths=lengths)
        for graph, res in graphs:
            res.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(res, eager)


def test_the_same_call_gives_the_same_bits():
    q, k, v = _inputs(1, 3, 20000, 8, 2, 128, seed=5)
    first = cr.attention(q, k, v)
    for _ in range(5):
        assert torch.equal(cr.attention(q, k, v), first)


def test_keys_beyond_four_gigabytes():
    # rows of 64 KB: key 65600 lies behind 2^32 bytes
    l, d = 66000, 64
    rows = torch.empty(l, 2 ** 15, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    k = rows[:, :d].unflatten(-1, (1, d))
    v = rows[:, -d:].unflatten(-1, (1, d))
    k.copy_(torch.randn(l, 1, d, generator=g, device=DEV))
    v.copy_(torch.randn(l, 1, d, generator=g, device=DEV))
    for m in (2, 200):
        q = torch.randn(m, 1, d, generator=g, device=DEV).to(torch.bfloat16)
        out = cr.attention(q, k, v)
        _check(q[None], k[None], v[None], out[None])
