"""Attention in the form where each wave has 32 queries of its own, for every size of heads, and masked heads of
every size in the other form: lengths around the blocks and tiles of keys, hidden keys, far scores, strides."""

import math

import pytest
import torch

import hadamard_rotated_int8_amd as cr
from kernel_names import launched
from test_gpu_attention import _check, _inputs

pytestmark = pytest.mark.gpu

SIZES = [64, 80, 128, 160, 192]  # of heads; the kernels are for 64, 96, 128, 160 and 192
KERNEL = {64: 64, 80: 96, 128: 128, 160: 160, 192: 192}
HEADS, M = 40, 257
AT = [0, 17, HEADS - 1]  # heads that are compared


def _own_queries(batch, kv, rows):
    """Whether the form with 32 queries to a wave is taken: more blocks of 32 rows than compute units."""
    return batch * kv * -(-rows // 32) > torch.cuda.get_device_properties(0).multi_processor_count


def _hidden(kind, batch, l, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kw = {}
    if kind in ("mask", "both"):
        kw["mask"] = torch.rand(batch, l, generator=g, device="cuda") < 0.6
        kw["mask"][:, l // 2] = True
    if kind in ("lengths", "both"):
        kw["lengths"] = torch.tensor([l - i * (l // 3) for i in range(batch)], dtype=torch.int32, device="cuda")
    return kw


def _check_heads(q, k, v, out, at=AT, ratio=1, **kw):
    key = [h // ratio for h in at]
    _check(q[:, :, at], k[:, :, key], v[:, :, key], out[:, :, at], **kw)


@pytest.mark.parametrize("kind", ["all", "lengths", "mask", "both"])
@pytest.mark.parametrize("l", [1, 31, 33, 63, 64, 65, 127, 129, 200])
@pytest.mark.parametrize("d", SIZES)
def test_own_queries(d, l, kind):
    assert _own_queries(1, HEADS, M)
    q, k, v = _inputs(1, M, l, HEADS, HEADS, d, seed=d + l)
    kw = _hidden(kind, 1, l, l)
    _check_heads(q, k, v, cr.attention(q, k, v, **kw), **kw)


@pytest.mark.parametrize("kind", ["all", "lengths", "mask", "both"])
@pytest.mark.parametrize("d", SIZES)
def test_own_queries_of_grouped_heads_and_a_batch(d, kind):
    batch, m, l, heads, kv = 2, 131, 333, 35, 7
    assert _own_queries(batch, kv, m * heads // kv)
    q, k, v = _inputs(batch, m, l, heads, kv, d, seed=d)
    kw = _hidden(kind, batch, l, d)
    _check_heads(q, k, v, cr.attention(q, k, v, **kw), [0, 4, 5, 34], heads // kv, **kw)


@pytest.mark.parametrize("kind", ["all", "both"])
@pytest.mark.parametrize("d", SIZES)
def test_own_queries_with_their_keys_split(d, kind):
    l = 1500
    q, k, v = _inputs(1, M, l, HEADS, HEADS, d, seed=d)
    kw = _hidden(kind, 1, l, d)
    out = cr.attention(q, k, v, **kw)
    _check_heads(q, k, v, out, **kw)
    assert "attention_join_kernel" in launched(lambda: cr.attention(q, k, v, **kw))[-1]


@pytest.mark.parametrize("bad", [math.nan, math.inf, torch.finfo(torch.bfloat16).min])
@pytest.mark.parametrize("d", SIZES)
def test_own_queries_hidden_keys_hold_anything(d, bad):
    l = 300
    q, k, v = _inputs(2, M, l, HEADS, HEADS, d, seed=d)
    k, v = k.clone(), v.clone()
    kw = _hidden("both", 2, l, d)
    clean = cr.attention(q, k, v, **kw)
    hidden = ~kw["mask"] | (torch.arange(l, device="cuda") >= kw["lengths"][:, None])
    k[hidden], v[hidden] = bad, bad
    assert torch.equal(cr.attention(q, k, v, **kw), clean)
    only = {"lengths": kw["lengths"]}
    k, v = k.nan_to_num(0, 0, 0).clamp(-4, 4), v.nan_to_num(0, 0, 0).clamp(-4, 4)
    clean = cr.attention(q, k, v, **only)
    behind = torch.arange(l, device="cuda") >= kw["lengths"][:, None]
    k[behind], v[behind] = bad, bad
    assert torch.equal(cr.attention(q, k, v, **only), clean)


@pytest.mark.parametrize("d", SIZES)
def test_own_queries_scores_far_apart_and_rising(d):
    l = 500
    q, k, v = _inputs(1, M, l, HEADS, HEADS, d, seed=7, scale_q=8.0)
    k = k * torch.linspace(0.1, 6, l, device="cuda")[None, :, None, None].to(torch.bfloat16)
    _check_heads(q, k, v, cr.attention(q, k, v))
    flipped = k.flip(1)
    _check_heads(q, flipped, v, cr.attention(q, flipped, v))
    ones = torch.ones_like(q)
    lift = (torch.arange(l, device="cuda").float() * 0.37)[None, :, None, None].expand(k.shape).to(torch.bfloat16)
    _check_heads(ones, lift, v, cr.attention(ones, lift, v))
    _check_heads(ones, -lift, v, cr.attention(ones, -lift, v))


@pytest.mark.parametrize("d", SIZES)
def test_own_queries_into_wider_rows(d):
    l = 130
    q, k, v = _inputs(2, M, l, HEADS, HEADS, d, seed=d)
    ref = cr.attention(q, k, v)
    wide = torch.full((2, HEADS, M + 3, d + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, :, 1:M + 1, 8:8 + d].transpose(1, 2)
    assert cr.attention(q, k, v, out=out) is out
    assert torch.equal(out, ref)
    out.fill_(7.0)
    assert (wide == 7.0).all()


@pytest.mark.parametrize("kind", ["mask", "both"])
@pytest.mark.parametrize("m, l", [(1, 33), (5, 100), (40, 257), (3, 2100)])
@pytest.mark.parametrize("d", SIZES)
def test_shared_queries_with_a_mask(d, m, l, kind):
    assert not _own_queries(2, 2, m)
    q, k, v = _inputs(2, m, l, 2, 2, d, seed=d + l)
    kw = _hidden(kind, 2, l, l)
    _check(q, k, v, cr.attention(q, k, v, **kw), **kw)


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("d", SIZES)
def test_which_kernels_these_are(d, masked):
    for m, heads, few in ((M, HEADS, False), (5, 2, True)):
        q, k, v = _inputs(1, m, 64, heads, heads, d)
        kw = _hidden("mask", 1, 64, 1) if masked else {}
        names = launched(lambda: cr.attention(q, k, v, **kw))
        assert names == [f"attention_kernel<{KERNEL[d]}, {str(few).lower()}, {str(masked).lower()}>"], names
