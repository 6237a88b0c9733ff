"""The ends of attention's range of scales: refused on the host, or right (the second on a GPU)."""

import pytest
import torch

import hadamard_rotated_int8_amd as cr
import test_attention_boundary as boundary


def test_scales_that_overflow_are_refused():
    assert boundary._apply(scale=2.3e38) == cr.OK
    for scale in (2.36e38, 3e38, 3.4e38):
        assert boundary._apply(scale=scale) == cr.ERR_UNSUPPORTED


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [1e-37, 1e-38, 1e-42])
@pytest.mark.parametrize("m, l, heads", [(5, 300, 2), (5, 2100, 2), (300, 300, 40)])
def test_vanishing_scales_take_the_mean(m, l, heads, scale):
    # weights are 1 within 2^-20, the scores' 40 times the scale: the mean of the values that are seen, off
    # by their sum's rounding and the output's of half a step, 2^-8; the first keys are hidden
    from test_gpu_attention import _inputs

    q, k, v = _inputs(1, m, l, heads, heads, 64, seed=l)
    mask = torch.ones(1, l, dtype=torch.bool, device="cuda")
    mask[:, :200] = False
    out = cr.attention(q, k, v, scale=scale, mask=mask)
    want = v[0, 200:].double().mean(0)
    tol = 2.0 ** -8 * want.abs() + l * 2.0 ** -23 * v[0, 200:].double().abs().mean(0)
    assert ((out[0].double() - want).abs() <= tol).all()


@pytest.mark.gpu
@pytest.mark.parametrize("m, l, heads", [(5, 300, 2), (5, 2100, 2), (300, 300, 40), (1500, 1100, 15)])
def test_vanishing_scales_beside_scores_of_minus_infinity(m, l, heads):
    # every other query's scores are minus infinity for the first keys, and vanish for the others
    from test_gpu_attention import _inputs

    q, k, v = _inputs(1, m, l, heads, heads, 64, seed=l)
    q, k = q.clone(), k.clone()
    cut = l * 2 // 5
    q[:, :, :, 3], k[:, :, :, 3] = 0, 0
    q[:, ::2, :, 3] = 3e38
    k[:, :cut, :, 3] = -3e38
    out = cr.attention(q, k, v, scale=1e-38)
    for first, at in ((cut, 0), (0, 1)):
        part = v[0, first:].double()
        tol = 2.0 ** -8 * part.mean(0).abs() + l * 2.0 ** -23 * part.abs().mean(0)
        assert ((out[0, at::2].double() - part.mean(0)).abs() <= tol).all()
