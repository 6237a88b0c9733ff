"""Attention where scores are minus infinity: weights of zero beside finite ones, and no softmax where all
that are seen are (GPU)."""

import pytest
import torch

import hadamard_rotated_int8_amd as cr
from test_gpu_attention import _check, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("d", [64, 80, 128, 160, 192])
# the waves of a workgroup on the same 32 queries, keys split or not; each on its own, the last tiles' keys split
@pytest.mark.parametrize("m, l, heads", [(5, 100, 2), (5, 2100, 2), (300, 70, 40), (1500, 1100, 15)])
def test_scores_of_minus_infinity(m, l, heads, d, masked):
    q, k, v = _inputs(3, m, l, heads, heads, d, seed=l + d)
    q, k = q.clone(), k.clone()
    mask = None
    if masked:
        mask = torch.rand(3, l, device="cuda", generator=torch.Generator(device="cuda").manual_seed(l)) < 0.5
        mask[:, l // 3] = True
    kw = {"mask": mask}
    q[:2, ::2], k[:2] = 0, 0
    q[:2, :, :, 3] = 0  # (1.2 times 3e38 would be infinite in the other queries)
    q[:2, ::2, :, 3] = 3e38
    k[0, :, :, 3] = -3e38  # all scores of every other query of entry 0 are minus infinity
    k[1, :, :, 3] = -3e38  # ... of entry 1 all but a few
    k[1, l // 3::l // 2, :, 3] = 0
    out = cr.attention(q, k, v, **kw)
    assert out[0, ::2].isnan().all()
    assert not out[0, 1::2].isnan().any() and not out[1:].isnan().any()
    # what the finite scores of those queries, which are 0, leave
    seen = torch.zeros(l, dtype=torch.bool, device="cuda")
    seen[l // 3::l // 2] = True
    if masked:
        seen &= mask[1]
    want = v[1, seen].double().mean(0)
    assert ((out[1, ::2].double() - want).abs() <= 2.0 ** -7 * v[1, seen].double().abs().amax(0)).all()
    at = [0, heads - 1]
    kw = {} if mask is None else {"mask": mask[2:]}
    _check(q[2:, :, at], k[2:, :, at], v[2:, :, at], out[2:, :, at], **kw)
