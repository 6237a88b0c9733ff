"""The float32 linear of two groups of waves asks for fragments before it waits for those before them (CPU).

In the K loop of fp8_gemm_kernel<1, 1, 2, 2, 2, 3> with power-of-two scales six of the eight 16-byte LDS reads
are on their way before the conversions of the third and fourth begin.  With the fifth and sixth behind that
wait it took 17.2 us instead of 16.6 at 48 x 5120 -> 13824.

Skipped when the library has not been built or there is no disassembler.
"""

import os
import re
import subprocess

import pytest

import test_code_objects as objects
from test_matrix_hazards import OBJDUMP

KERNEL = "fp8_gemm_kernelILi1ELi1ELi2ELi2ELi2ELi3ELb0ELb1ELb0EE"


def _reads_ahead(lines):
    """How many 16-byte reads stand in front of the second wait for LDS that has conversions right behind it."""
    at = [i for i, ln in enumerate(lines) if ln.startswith("v_mfma")]
    start = max(i for i, ln in enumerate(lines[:at[0]]) if ln.startswith("s_barrier"))
    reads, waits, converting = 0, 0, False
    for ln in lines[start:]:
        if ln.startswith("ds_read_b128"):
            reads += 1
        elif ln.startswith("s_waitcnt") and "lgkmcnt" in ln:
            converting = False
        elif ln.startswith("v_cvt_scalef32") and not converting:
            converting, waits = True, waits + 1
            if waits == 2:
                return reads
    return reads


def test_the_count():
    cvt, read, wait, mfma = "v_cvt_scalef32_pk_bf16_fp8 v0, v1, v2", "ds_read_b128 v[0:3], v9", \
        "s_waitcnt lgkmcnt(0)", "v_mfma_f32_32x32x16_bf16 a[0:15], v[0:3], v[4:7], a[0:15]"
    head = ["s_barrier"] + [read] * 4 + [wait, cvt, cvt, mfma]
    assert _reads_ahead(head + [read, read, wait, cvt, mfma]) == 6
    assert _reads_ahead(head + [wait, cvt, read, read, mfma]) == 4


def test_built_code(tmp_path):
    lib = objects.LIBS[0]
    if not os.path.exists(lib):
        pytest.skip("libconvrot.so not built")
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump")
    found = 0
    for n, (_, code) in enumerate(objects._device_code_objects(open(lib, "rb").read())):
        if not any(KERNEL in k[".name"] for k in objects._kernels(code)):
            continue
        path = tmp_path / f"{n}.co"
        path.write_bytes(code)
        text = subprocess.run([OBJDUMP, "-d", "--mcpu=gfx950", str(path)], capture_output=True, text=True,
                              check=True).stdout
        body = re.search(rf"<[^>]*{KERNEL}[^>]*>:\n(.*?)(?:\n\n|\Z)", text, re.S)[1]
        lines = [ln.split("//")[0].strip() for ln in body.splitlines()]
        assert _reads_ahead([ln for ln in lines if ln]) == 6
        found += 1
    assert found == 1
