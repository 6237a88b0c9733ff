"""Rotary positions against a plain 64-bit reference (GPU).

Tolerances.  The angle is formed in float64, reduced to a fraction of a turn
and rounded to float32 once: the fraction (at most 1/2) is off by 2^-25 of a
turn, the angle by 2 pi 2^-25, and sine and cosine by at most 4 more float32
roundings (2 ulp each of the function, the factor's product), 2^-22 in all.
A result a c - b s has two products and one rounding: |error| <= (2^-22 +
2^-23) factor (|a| + |b|), plus half a step of the output's type
(finfo.eps / 2 of the value: 2^-24 and 2^-8).  The
float64 product of position and frequency (each with a rounding of 2^-53)
adds 2^-51 angle, below 2^-22 for angles up to 2^28.
"""

import pytest
import torch

import block_reference as ref
import hadamard_rotated_int8_amd as cr

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    cr.lib()
    yield
    torch.cuda.synchronize()


def _x(*shape, dtype=torch.float32, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def _partner(x, plan):
    """|a| + |b| for each rotated feature (zero elsewhere)."""
    rot, s = 2 * plan.inv_freq.numel(), plan.start
    out = torch.zeros(x.shape, dtype=torch.float64)
    p = x.cpu().double()[..., s:s + rot].abs()
    if plan.layout == "half":
        t = p[..., :rot // 2] + p[..., rot // 2:]
        out[..., s:s + rot] = torch.cat([t, t], -1)
    else:
        out[..., s:s + rot] = (p[..., 0::2] + p[..., 1::2]).repeat_interleave(2, -1)
    return out


def _check(y, x, plan, positions, inverse=False):
    want = ref.rope(x, plan.inv_freq, plan.layout, positions, plan.axis, plan.factor, plan.start, inverse)
    tol = 1.5 * 2.0 ** -22 * plan.factor * _partner(x, plan) + HALF_STEP[y.dtype] * want.abs()
    assert y.shape == x.shape
    assert bool(((y.cpu().double() - want).abs() <= tol + 1e-37).all())


DIMS = [(2, 2, 0), (8, 4, 2), (40, 40, 0), (64, 64, 0), (96, 64, 32), (128, 128, 0), (128, 50, 3),
        (80, 20, 60), (130, 126, 1), (256, 256, 0), (4096, 4096, 0)]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot,start", DIMS)
@pytest.mark.parametrize("xt,yt", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                   (torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)])
def test_rope(d, rot, start, layout, xt, yt):
    tokens, heads = (37, 5) if d < 1000 else (3, 2)
    print(f"[gpu] rope d={d} rot={rot} start={start} {layout} {xt}->{yt}", flush=True)
    plan = cr.rope_plan(rot, layout=layout, start=start)
    x = _x(tokens, heads, d, dtype=xt, seed=d)
    pos = torch.arange(100, 100 + tokens)
    y = cr.rope(x.cuda(), plan, pos.cuda(), out_dtype=yt)
    assert y.dtype == yt
    _check(y, x, plan, pos)


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64, torch.float32])
def test_far_and_fractional_positions(dtype):
    plan = cr.rope_plan(64)
    pos = torch.tensor([0, 1, -5, 4095, 131071, 1000003, 16777213], dtype=dtype)
    if dtype == torch.float32:
        pos = pos + 0.375 * (pos.abs() < 1e6)
    x = _x(7, 3, 64)
    _check(cr.rope(x.cuda(), plan, pos.cuda()), x, plan, pos)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_axes_batch_and_query_groups(layout):
    """Three positions per token, its own positions for each sequence, and more query than key heads
    in one launch, from column ranges of one buffer."""
    plan = cr.rope_plan(44, layout=layout, axes=(16, 14, 14), start=2)
    rows = _x(2, 33, 10, 48, dtype=torch.bfloat16).cuda()
    q, k = rows[:, :, :8], rows[:, :, 8:]
    pos = torch.randint(0, 500, (2, 33, 3), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    yq, yk = cr.rope([q, k], plan, pos.cuda(), out_dtype=torch.float32)
    _check(yq, q, plan, pos)
    _check(yk, k, plan, pos)
    # positions shared by the batch
    yq, yk = cr.rope([q, k], plan, pos[0].cuda())
    _check(yq, q, plan, pos[0])
    _check(yk, k, plan, pos[0])


def test_head_major_views_and_single_tokens():
    """[batch, heads, tokens, d] storage through a transposed view, odd row offsets, one token."""
    plan = cr.rope_plan(32, layout="half")
    store = _x(2, 4, 9, 33, dtype=torch.bfloat16).cuda()
    x = store.transpose(1, 2)[..., 1:]  # [batch, tokens, heads, 32], rows 33 apart
    pos = torch.arange(9, device="cuda")
    y = cr.rope(x, plan, pos)
    _check(y, x.cpu(), plan, pos)
    one = x[:1, 4:5]
    _check(cr.rope(one, plan, pos[4:5]), one.cpu(), plan, pos[4:5])


def test_in_place_and_back():
    """In place, the features beside the slice and the other rows stay; inverse turns back."""
    plan = cr.rope_plan(24, start=4)
    buf = _x(50, 3, 40).cuda()
    kept = buf.clone()
    x = buf[::2, :, 2:34]
    pos = torch.arange(25, device="cuda") * 7
    want = cr.rope(x, plan, pos)
    assert cr.rope(x, plan, pos, out=x) is x
    assert torch.equal(x, want)
    back = cr.rope(want, plan, pos, inverse=True)
    _check(back, want.cpu(), plan, pos, inverse=True)
    moved = kept[::2, :, 2:34]
    assert (back - moved).abs().max() <= 16 * 2.0 ** -23 * moved.abs().max()
    kept[::2, :, 2:34] = want
    assert torch.equal(buf, kept)


@pytest.mark.parametrize("scaling", [
    {"type": "linear", "factor": 4.0}, {"type": "ntk", "factor": 8.0},
    {"type": "yarn", "factor": 16.0, "original_length": 4096},
    {"type": "factors", "factors": [1.0 + 0.25 * i for i in range(32)], "attention_factor": 1.2}])
def test_scaled_frequencies(scaling):
    plan = cr.rope_plan(64, layout="half", scaling=scaling)
    x = _x(11, 2, 64)
    pos = torch.arange(11) * 9973
    _check(cr.rope(x.cuda(), plan, pos.cuda()), x, plan, pos)


def test_pairs_at_infinity_stay_alone():
    plan = cr.rope_plan(32)
    x = _x(4, 2, 32)
    x[1, 0, 4] = float("inf")
    x[2, 1, 9] = float("nan")
    pos = torch.arange(4)
    y = cr.rope(x.cuda(), plan, pos.cuda()).cpu()
    bad = torch.zeros(x.shape, dtype=torch.bool)
    bad[1, 0, 4:6] = True
    bad[2, 1, 8:10] = True
    assert torch.isfinite(y[~bad]).all() and not torch.isfinite(y[bad]).any()


def test_empty_calls():
    plan = cr.rope_plan(32)
    assert cr.rope(torch.empty(0, 4, 32, device="cuda"), plan,
                   torch.empty(0, dtype=torch.int32, device="cuda")).shape == (0, 4, 32)
    q, k = cr.rope([torch.ones(2, 0, 32, device="cuda"), torch.ones(2, 1, 32, device="cuda")], plan,
                   torch.tensor([0, 0], device="cuda"))
    assert q.shape == (2, 0, 32) and (k == 1).all()


def test_axes_that_positions_do_not_have():
    """Too few positions for the plan are refused; a pair that names an axis outside them has no
    position: its results are NaN, the others stay."""
    plan = cr.rope_plan(12, axes=(4, 4, 4))
    x = _x(5, 2, 12).cuda()
    pos = torch.arange(10, device="cuda").view(5, 2)
    with pytest.raises(ValueError, match="axes"):
        cr.rope(x, plan, pos)
    for bad in (2, -1):
        own = cr.RopePlan(plan.inv_freq, axis=torch.tensor([0, 0, 1, 1, bad, 0], dtype=torch.int32).cuda())
        y = cr.rope(x, own, pos)
        assert torch.isnan(y[..., 8:10]).all()
        good = cr.RopePlan(plan.inv_freq, axis=torch.tensor([0, 0, 1, 1, 0, 0], dtype=torch.int32).cuda())
        want = cr.rope(x, good, pos)
        assert torch.equal(y[..., :8], want[..., :8]) and torch.equal(y[..., 10:], want[..., 10:])
