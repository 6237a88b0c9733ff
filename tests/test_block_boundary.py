"""C-ABI refusals of the FP8 linears, the block norms and the rotary positions (no GPU needed), and
the frequencies of the rotary plans.

The library validates every argument on the host before any HIP call: each
call below fails validation, so none launches a kernel.
"""

import ctypes
import math
import struct

import pytest
import torch

import hadamard_rotated_int8_amd as cr
from hadamard_rotated_int8_amd import block

# Fake device addresses: only where no GPU is visible.
cpu_only = pytest.mark.skipif(
    torch.cuda.is_available(),
    reason="passes fake device pointers; host-validation tests run on GPU-less hosts only")

FAKE = 0x10000
NULL, SHAPE, DTYPE, UNSUPPORTED = cr.ERR_NULL, cr.ERR_SHAPE, cr.ERR_DTYPE, cr.ERR_UNSUPPORTED
BIG = 1 << 31


def _buffer(b):
    return ctypes.create_string_buffer(b, len(b))


# ---------------------------------------------------------------- FP8 linears

def _pack(x=FAKE, dt=cr.BF16, m=4, k=256, ldx=256, q=FAKE, scale=FAKE, lds=4, out=True):
    p = _buffer(block._FP8_PACKED.pack(q, scale, 0, 0, lds)) if out else None
    return cr.lib().convrot_fp8_pack_activations(x, dt, m, k, ldx, p, None)


@cpu_only
@pytest.mark.parametrize("want,args", [
    (NULL, dict(out=False)), (NULL, dict(x=None)), (NULL, dict(q=0)), (NULL, dict(scale=0)),
    (SHAPE, dict(k=0)), (SHAPE, dict(k=cr.MAX_K + 16, ldx=cr.MAX_K + 16)), (SHAPE, dict(m=-1)),
    (SHAPE, dict(m=BIG)), (SHAPE, dict(ldx=240)), (SHAPE, dict(ldx=1 << 41)), (SHAPE, dict(lds=3)),
    (DTYPE, dict(dt=cr.I32)), (DTYPE, dict(dt=cr.E8M0)), (DTYPE, dict(dt=-1)),
    (UNSUPPORTED, dict(k=248, ldx=248)), (UNSUPPORTED, dict(ldx=260)), (UNSUPPORTED, dict(x=FAKE + 2)),
    (UNSUPPORTED, dict(q=FAKE + 8)), (UNSUPPORTED, dict(scale=FAKE + 2)), (UNSUPPORTED, dict(lds=6))])
def test_fp8_pack_refusals(want, args):
    assert _pack(**args) == want


@cpu_only
@pytest.mark.parametrize("want,args", [
    (NULL, dict(w=None)), (NULL, dict(q=None)), (NULL, dict(s=None)), (SHAPE, dict(k=0)),
    (SHAPE, dict(n=-1)), (SHAPE, dict(n=BIG)), (SHAPE, dict(ld=100)),
    (SHAPE, dict(n=BIG - 1, k=131072, ld=131072)), (DTYPE, dict(dt=7)), (UNSUPPORTED, dict(k=136, ld=136)),
    (UNSUPPORTED, dict(w=FAKE + 2)), (UNSUPPORTED, dict(q=FAKE + 4))])
def test_fp8_weight_refusals(want, args):
    a = dict(w=FAKE, dt=cr.F32, n=64, k=128, ld=128, q=FAKE, s=FAKE) | args
    assert cr.lib().convrot_fp8_quantize_weights(a["w"], a["dt"], a["n"], a["k"], a["ld"], a["q"], a["s"],
                                                 None) == want


def _linear(x=True, q=FAKE, scale=FAKE, m=4, k=256, lds=4, ws=None, count=None, y=(FAKE,), ldy=(64,),
            ydt=cr.F32, act=cr.ACT_NONE):
    ws = ws or [{}]
    packed = b"".join(block._FP8_WEIGHTS.pack(*(
        (dict(q=FAKE, s=FAKE, b=0, n=64, k=256, dt=cr.E8M0) | w).values())) for w in ws)
    p = block._FP8_PACKED.pack(q, scale, m, k, lds) if x else None
    return cr.lib().convrot_fp8_linear_grouped(
        p, packed, len(ws) if count is None else count, struct.pack(f"={len(y)}Q", *y),
        struct.pack(f"={len(ldy)}q", *ldy), ydt, act, None)


@cpu_only
@pytest.mark.parametrize("want,args", [
    (NULL, dict(x=False)), (NULL, dict(q=0)), (NULL, dict(scale=0)), (NULL, dict(y=(0,))),
    (NULL, dict(ws=[dict(q=0)])), (NULL, dict(ws=[dict(s=0)])),
    (SHAPE, dict(count=0)), (SHAPE, dict(count=9)), (SHAPE, dict(k=0)), (SHAPE, dict(m=-1)),
    (SHAPE, dict(m=BIG, lds=BIG)), (SHAPE, dict(lds=0)), (SHAPE, dict(ldy=(63,))),
    (SHAPE, dict(ws=[dict(k=128)])), (SHAPE, dict(ws=[dict(n=-1)])), (SHAPE, dict(ws=[dict(n=BIG)])),
    (SHAPE, dict(m=BIG - 1, lds=BIG, ws=[dict(n=BIG - 1)], ldy=(BIG,))),
    (DTYPE, dict(ydt=cr.I32)), (DTYPE, dict(act=2)), (DTYPE, dict(ws=[dict(dt=cr.BF16)])),
    (DTYPE, dict(ws=[dict(), dict(dt=cr.F32)], y=(FAKE, FAKE), ldy=(64, 64))),
    (UNSUPPORTED, dict(k=264, ws=[dict(k=264)])), (UNSUPPORTED, dict(lds=6)),
    (UNSUPPORTED, dict(q=FAKE + 8)), (UNSUPPORTED, dict(scale=FAKE + 1)),
    (UNSUPPORTED, dict(ws=[dict(q=FAKE + 8)])), (UNSUPPORTED, dict(ws=[dict(s=FAKE + 2, dt=cr.F32)])),
    (UNSUPPORTED, dict(ws=[dict(b=FAKE + 2)])), (UNSUPPORTED, dict(y=(FAKE + 2,))),
    (UNSUPPORTED, dict(y=(FAKE + 1,), ydt=cr.BF16))])
def test_fp8_linear_refusals(want, args):
    assert _linear(**args) == want


def _linear_rows(x=FAKE, dt=cr.BF16, m=4, k=256, ldx=256, n=64, wk=256, q=FAKE, y=FAKE, ldy=64, ydt=cr.F32,
                 act=cr.ACT_NONE, count=1):
    return cr.lib().convrot_fp8_linear_rows(
        x, dt, m, k, ldx, block._FP8_WEIGHTS.pack(q, FAKE, 0, n, wk, cr.E8M0), count, struct.pack("=Q", y),
        struct.pack("=q", ldy), ydt, act, None)


@cpu_only
@pytest.mark.parametrize("want,args", [
    (NULL, dict(x=None)), (NULL, dict(q=0)), (NULL, dict(y=0)), (SHAPE, dict(m=17)), (SHAPE, dict(m=-1)),
    (SHAPE, dict(k=-16)), (SHAPE, dict(k=2 ** 63 - 1)), (SHAPE, dict(k=cr.MAX_K + 16)),
    (SHAPE, dict(m=2, k=24592, wk=24592, ldx=24592)), (SHAPE, dict(ldx=255)), (SHAPE, dict(wk=128)), (SHAPE, dict(ldy=63)), (SHAPE, dict(count=0)),
    (DTYPE, dict(dt=cr.I32)), (DTYPE, dict(ydt=cr.I32)), (DTYPE, dict(act=3)),
    (UNSUPPORTED, dict(x=FAKE + 8)), (UNSUPPORTED, dict(ldx=260)), (UNSUPPORTED, dict(k=264, wk=264, ldx=264))])
def test_fp8_linear_rows_refusals(want, args):
    assert _linear_rows(**args) == want


@cpu_only
def test_fp8_empty_calls_launch_nothing():
    assert _linear_rows(m=0, x=None, q=0, y=0) == cr.OK
    assert _pack(m=0, x=None, q=0, scale=0) == cr.OK
    assert _linear(m=0, q=0, scale=0, y=(0,), ws=[dict(q=0, s=0)]) == cr.OK
    assert _linear(ws=[dict(n=0, q=0, s=0)], y=(0,), q=0, scale=0) == cr.OK


# ---------------------------------------------------------------- block norms

def _vec(data=0, stride=0, rows=1, dt=cr.F32):
    return data, stride, rows, dt


def _norm(kind=0, eps=1e-6, weight=_vec(), bias=_vec()):
    return kind, eps, *weight, *bias


def _block(x=FAKE, branch=0, h=0, y=FAKE, packed=None, m=4, k=64, ldx=64, ldb=64, ldh=64, ldy=64,
           xdt=cr.BF16, bdt=cr.F32, ydt=cr.BF16, rs=1.0, gate=_vec(), scale=_vec(), shift=_vec(),
           post=_norm(), pre=_norm(2)):
    p = _buffer(block._FP8_PACKED.pack(*packed)) if packed else None
    return cr.lib().convrot_block_norm(block._BLOCK.pack(
        x, branch, h, y, ctypes.addressof(p) if p else 0, m, k, ldx, ldb, ldh, ldy, xdt, bdt, ydt, rs,
        *gate, *scale, *shift, *post, *pre), None)


PACKED = (FAKE, FAKE, 0, 0, 4)


@cpu_only
@pytest.mark.parametrize("want,args", [
    (NULL, dict(x=0)), (NULL, dict(y=0, pre=_norm())), (NULL, dict(y=0, packed=(0, FAKE, 0, 0, 4))),
    (SHAPE, dict(k=0)), (SHAPE, dict(k=32769, ldx=40000, ldy=40000)), (SHAPE, dict(m=-1)),
    (SHAPE, dict(m=BIG)), (SHAPE, dict(ldx=63)), (SHAPE, dict(ldy=63)),
    (SHAPE, dict(branch=FAKE, ldb=63)), (SHAPE, dict(branch=FAKE, h=FAKE, ldh=63)),
    (SHAPE, dict(scale=_vec(FAKE, -1))), (SHAPE, dict(shift=_vec(FAKE, 0, 0))),
    (SHAPE, dict(y=0, packed=(FAKE, FAKE, 0, 0, 0))),
    (DTYPE, dict(xdt=cr.I32)), (DTYPE, dict(ydt=cr.E8M0)), (DTYPE, dict(branch=FAKE, bdt=2)),
    (DTYPE, dict(scale=_vec(FAKE, dt=2))), (DTYPE, dict(pre=_norm(3))),
    (DTYPE, dict(branch=FAKE, post=_norm(-1))), (DTYPE, dict(pre=_norm(1, weight=_vec(FAKE, dt=5)))),
    (UNSUPPORTED, dict(packed=PACKED)),                       # y and packed
    (UNSUPPORTED, dict(h=FAKE)), (UNSUPPORTED, dict(gate=_vec(FAKE))), (UNSUPPORTED, dict(rs=0.5)),
    (UNSUPPORTED, dict(post=_norm(1))),                       # these need a branch
    (UNSUPPORTED, dict(y=0, branch=FAKE, h=FAKE)),            # a norm of a y that is not wanted
    (UNSUPPORTED, dict(y=0, branch=FAKE, h=FAKE, pre=_norm(), scale=_vec(FAKE))),
    (UNSUPPORTED, dict(pre=_norm(0, weight=_vec(FAKE)))),     # a weight without a norm
    (UNSUPPORTED, dict(pre=_norm(1, eps=-1.0))), (UNSUPPORTED, dict(pre=_norm(2, eps=math.nan))),
    (UNSUPPORTED, dict(x=FAKE + 1)), (UNSUPPORTED, dict(y=FAKE + 2, ydt=cr.F32)),
    (UNSUPPORTED, dict(branch=FAKE + 2)), (UNSUPPORTED, dict(scale=_vec(FAKE + 2))),
    (UNSUPPORTED, dict(y=0, packed=PACKED, k=56)), (UNSUPPORTED, dict(y=0, packed=(FAKE + 8, FAKE, 0, 0, 4))),
    (UNSUPPORTED, dict(ldy=128)), (UNSUPPORTED, dict(ydt=cr.F32)),   # over x, but not row by row
    (UNSUPPORTED, dict(y=0, branch=FAKE + 64, h=FAKE, ldh=128, pre=_norm())),
    (UNSUPPORTED, dict(branch=FAKE + 64, h=FAKE + 128, y=FAKE + 128)), (UNSUPPORTED, dict(branch=FAKE + 64, h=FAKE)),
    (UNSUPPORTED, dict(branch=FAKE + 64, h=FAKE + 64)), (UNSUPPORTED, dict(branch=FAKE + 64, y=FAKE + 64)),
    (UNSUPPORTED, dict(y=0, packed=(FAKE, FAKE + 1, 0, 0, 4))), (UNSUPPORTED, dict(y=0, packed=(FAKE, FAKE, 0, 0, 5)))])
def test_block_norm_refusals(want, args):
    assert _block(**args) == want


@cpu_only
def test_block_norm_null_and_empty():
    assert cr.lib().convrot_block_norm(None, None) == NULL
    assert _block(m=0, x=0, y=0) == cr.OK


# ------------------------------------------------------------ rotary positions

def _rope(inv=FAKE, axis=0, pos=FAKE, ps=(0, 1), batch=1, tokens=4, pdt=0, d=64, rot=64, start=0,
          layout=0, xdt=cr.BF16, ydt=cr.BF16, count=1, axes=1, t=None):
    t = t or [{}]
    tensors = []
    for one in t:
        o = dict(x=FAKE, y=FAKE + 0x1000, xs=(0, 128, 64), ys=(0, 128, 64), heads=2) | one
        tensors += [o["x"], o["y"], *o["xs"], *o["ys"], o["heads"]]
    tensors += [0] * (36 - len(tensors))
    return cr.lib().convrot_rope_apply(block._ROPE.pack(
        inv, axis, pos, *ps, batch, tokens, pdt, d, rot, start, layout, 0, xdt, ydt, 1.0, count, axes, *tensors),
        None)


@cpu_only
@pytest.mark.parametrize("want,args", [
    (NULL, dict(inv=0)), (NULL, dict(pos=0)), (NULL, dict(t=[dict(x=0)])), (NULL, dict(t=[dict(y=0)])),
    (SHAPE, dict(count=0)), (SHAPE, dict(count=5)), (SHAPE, dict(axes=0)), (SHAPE, dict(batch=-1)), (SHAPE, dict(tokens=BIG)),
    (SHAPE, dict(batch=1 << 16, tokens=1 << 16)), (SHAPE, dict(rot=63)), (SHAPE, dict(rot=0)),
    (SHAPE, dict(rot=66)), (SHAPE, dict(rot=32, start=33)), (SHAPE, dict(rot=32, start=-1)),
    (SHAPE, dict(d=4098, rot=64)), (SHAPE, dict(d=1)), (SHAPE, dict(ps=(-1, 1))), (SHAPE, dict(ps=(0, 1 << 41))),
    (SHAPE, dict(t=[dict(heads=-1)])), (SHAPE, dict(t=[dict(heads=4097)])),
    (SHAPE, dict(d=128, t=[dict(heads=2049)])), (SHAPE, dict(t=[dict(xs=(0, -1, 64))])),
    (SHAPE, dict(t=[dict(ys=(1 << 41, 1, 64))])),
    (DTYPE, dict(xdt=2)), (DTYPE, dict(ydt=3)), (DTYPE, dict(pdt=3)), (DTYPE, dict(pdt=-1)),
    (DTYPE, dict(layout=2)),
    (UNSUPPORTED, dict(inv=FAKE + 4)), (UNSUPPORTED, dict(axis=FAKE + 2)), (UNSUPPORTED, dict(pos=FAKE + 4, pdt=1)),
    (UNSUPPORTED, dict(t=[dict(x=FAKE + 1)])), (UNSUPPORTED, dict(ydt=cr.F32, t=[dict(y=FAKE + 2)])),
    (UNSUPPORTED, dict(ydt=cr.F32, t=[dict(y=FAKE)])),                        # in place, another type
    (UNSUPPORTED, dict(t=[dict(y=FAKE, ys=(0, 256, 64))]))])                  # in place, other strides
def test_rope_refusals(want, args):
    assert _rope(**args) == want


@cpu_only
def test_rope_null_and_empty():
    assert cr.lib().convrot_rope_apply(None, None) == NULL
    assert _rope(tokens=0, t=[dict(x=0, y=0)]) == cr.OK
    assert _rope(t=[dict(x=0, y=0, heads=0)], inv=0, pos=0) == cr.OK


# ------------------------------------------------------------ the Python layer

def test_host_tensors_are_refused():
    x = torch.zeros(4, 128)
    w = cr.Fp8Weights(torch.zeros(8, 128).to(torch.float8_e4m3fn), torch.ones(1, 1))
    plan = cr.rope_plan(64, device="cpu")
    for call in (lambda: cr.fp8_pack_activations(x), lambda: cr.fp8_quantize_weights(x),
                 lambda: cr.fp8_linear(x, w), lambda: cr.block_norm(x, cr.Norm("rms")),
                 lambda: cr.block_update(x, x), lambda: cr.rope(x.view(4, 2, 64), plan, torch.arange(4))):
        with pytest.raises(ValueError, match="device tensor"):
            call()


def test_rope_plan_frequencies():
    p = cr.rope_plan(8, theta=10000.0, device="cpu")
    assert p.inv_freq.dtype == torch.float64 and p.axis is None and p.factor == 1.0
    want = torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64)
    assert torch.allclose(p.inv_freq, want, rtol=1e-14)
    p = cr.rope_plan(8, axes=(4, 2, 2), device="cpu")
    assert p.axis.tolist() == [0, 0, 1, 2]
    assert torch.allclose(p.inv_freq, torch.tensor([1.0, 0.01, 1.0, 1.0], dtype=torch.float64), rtol=1e-14)
    p = cr.rope_plan(8, scaling={"type": "linear", "factor": 4.0}, device="cpu")
    assert torch.allclose(p.inv_freq, want / 4, rtol=1e-14)
    # the first pair keeps its frequency, the last is slowed by exactly the factor
    p = cr.rope_plan(8, scaling={"type": "ntk", "factor": 4.0}, device="cpu")
    assert math.isclose(p.inv_freq[0], 1.0) and math.isclose(p.inv_freq[-1], want[-1] / 4, rel_tol=1e-12)
    p = cr.rope_plan(64, scaling={"type": "yarn", "factor": 4.0, "original_length": 2048}, device="cpu")
    plain = cr.rope_plan(64, device="cpu").inv_freq
    turns = 2048 * plain / (2 * math.pi)
    assert torch.equal(p.inv_freq[turns > 32 * 1.4], plain[turns > 32 * 1.4])
    assert torch.allclose(p.inv_freq[turns < 1 / 1.4], plain[turns < 1 / 1.4] / 4, rtol=1e-14)
    between = (turns < 32 / 1.4) & (turns > 1.4)
    assert between.any() and (p.inv_freq[between] < plain[between]).all()
    assert (p.inv_freq[between] > plain[between] / 4).all()
    assert math.isclose(p.factor, 0.1 * math.log(4.0) + 1)
    p = cr.rope_plan(4, scaling={"type": "factors", "factors": [1.0, 5.0], "attention_factor": 1.1}, device="cpu")
    assert torch.allclose(p.inv_freq, torch.tensor([1.0, 0.002], dtype=torch.float64), rtol=1e-14)
    assert p.factor == 1.1


@pytest.mark.parametrize("args", [
    dict(rot=7), dict(rot=0), dict(rot=8, start=-1), dict(rot=8, layout="whole"), dict(rot=8, theta=1.0),
    dict(rot=8, axes=(4, 2)), dict(rot=8, axes=(5, 3)), dict(rot=8, scaling={"type": "other"}),
    dict(rot=8, scaling={"type": "linear", "factor": 0.5}), dict(rot=8, scaling={"type": "linear", "more": 1}),
    dict(rot=8, scaling={"type": "factors", "factors": [1.0]}),
    dict(rot=8, scaling={"type": "factors", "factors": [1.0, 1.0, 0.0, 1.0]}),
    dict(rot=8, axes=(4, 4), scaling={"type": "ntk", "factor": 2.0}),
    dict(rot=8, scaling={"type": "yarn", "factor": 2.0, "original_length": 0})])
def test_rope_plan_refusals(args):
    with pytest.raises(ValueError):
        cr.rope_plan(device="cpu", **args)


def test_struct_formats_have_the_header_s_sizes(tmp_path):
    """The formats the binding packs are as long as the C compiler's structs."""
    import shutil
    import subprocess

    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    import os

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "convrot.h"\n'
                   'int main(void) { printf("%zu %zu %zu %zu %zu %zu", sizeof(convrot_fp8_packed), '
                   'sizeof(convrot_fp8_weights), sizeof(convrot_block), sizeof(convrot_rope), '
                   'offsetof(convrot_block, post), offsetof(convrot_rope, t)); return 0; }\n')
    exe = tmp_path / "sizes"
    subprocess.run([cc, "-I", os.path.join(root, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    assert got == [block._FP8_PACKED.size, block._FP8_WEIGHTS.size, block._BLOCK.size, block._ROPE.size,
                   struct.calcsize("=5Q6q3if" + 3 * block._VECTOR), struct.calcsize("=3Q4q8ifii4x")]
