"""Attention of queries that see no key: zeros, whatever the queries hold (GPU)."""

import math

import pytest
import torch

import hadamard_rotated_int8_amd as cr
from test_gpu_attention import _check, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("d", [64, 80, 128, 160, 192])
# the waves of a workgroup on the same 32 queries, keys split or not; each on its own, the last tiles' keys split
@pytest.mark.parametrize("batch, m, l, heads", [(3, 5, 100, 2), (3, 5, 2100, 2), (3, 300, 70, 40), (3, 1500, 1100, 15)])
def test_a_query_that_sees_no_key_gives_zeros(batch, m, l, heads, d, bad):
    q, k, v = _inputs(batch, m, l, heads, heads, d, seed=l + d)
    mask = torch.rand(batch, l, device="cuda", generator=torch.Generator(device="cuda").manual_seed(l)) < 0.5
    mask[1] = False
    clean = cr.attention(q, k, v, mask=mask)
    q = q.clone()
    q[1, ::3, :, d - 1] = bad
    out = cr.attention(q, k, v, mask=mask)
    assert (out[1] == 0).all()
    assert torch.equal(out[0], clean[0]) and torch.equal(out[2], clean[2])
    heads_checked = [0, heads - 1]
    _check(q[2:, :, heads_checked], k[2:, :, heads_checked], v[2:, :, heads_checked], out[2:, :, heads_checked],
           mask=mask[2:])
    lengths = torch.tensor([l, 0, l // 2], dtype=torch.int32, device="cuda")
    assert (cr.attention(q, k, v, lengths=lengths)[1] == 0).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("m, l, heads", [(5, 100, 2), (5, 2100, 2), (300, 70, 40)])
def test_a_query_that_sees_one_key_keeps_its_nan(m, l, heads, bad):
    q, k, v = _inputs(2, m, l, heads, heads, 64, seed=l)
    mask = torch.zeros(2, l, dtype=torch.bool, device="cuda")
    mask[1, l - 1] = True
    q = q.clone()
    q[:, 0, :, 0] = bad
    out = cr.attention(q, k, v, mask=mask)
    assert (out[0] == 0).all() and out[1, 0].isnan().all()
    assert torch.equal(out[1, 1:], v[1, l - 1].expand_as(out[1, 1:]))
