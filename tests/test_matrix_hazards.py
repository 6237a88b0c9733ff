"""Matrix instructions written as inline assembly keep the distances the hardware needs (CPU).

The compiler inserts wait states around the matrix instructions it knows; it
does not see those inside inline assembly (fp8_gemm_wide.hip).  The built
gfx950 code is disassembled and every v_mfma_scale of its kernels checked:

* no vector instruction writes one of its operands less than 2 wait states
  before it;
* no instruction touches a result held in vector registers before two more
  matrix instructions (32 cycles each) or 11 wait states have passed.

Skipped when the library has not been built or there is no disassembler.
"""

import os
import re
import shutil
import subprocess

import pytest

import test_code_objects as objects

OBJDUMP = shutil.which("llvm-objdump") or "/opt/rocm/llvm/bin/llvm-objdump"


def _registers(text):
    out = set()
    for lo, hi, one in re.findall(r"\bv\[(\d+):(\d+)\]|\bv(\d+)\b", text):
        out |= {int(one)} if one else set(range(int(lo), int(hi) + 1))
    return out


def _wait_states(ins):
    return 1 + int(ins.split()[1], 0) if ins.startswith("s_nop") else 1


def _hazards(lines):
    """(checked, descriptions) for the instructions of one kernel, in order."""
    found, checked = [], 0
    for k, ins in enumerate(lines):
        if not ins.startswith("v_mfma_scale"):
            continue
        checked += 1
        result, operands = ins.split(None, 1)[1].split(",", 1)
        sources, states, j = _registers(operands), 0, k - 1
        while j >= 0 and states < 2:
            prev = lines[j]
            if prev.startswith("v_") and not prev.startswith(("v_mfma", "v_cmp")) and \
                    _registers(prev.split(None, 1)[1].split(",")[0]) & sources:
                found.append(f"{prev} -> {ins}")
            states += _wait_states(prev)
            j -= 1
        held, later, states, j = _registers(result), 0, 0, k + 1
        while held and j < len(lines) and later < 2 and states < 11:
            nxt = lines[j]
            if nxt.startswith("v_mfma"):
                later += 1
            elif nxt.startswith("s_nop"):
                states += _wait_states(nxt)
            elif nxt.startswith(("v_", "ds_", "buffer_", "global_", "scratch_", "flat_")) and \
                    _registers(nxt.split(None, 1)[1]) & held:
                found.append(f"{ins} <- {nxt}")
            j += 1
    return checked, found


def test_a_planted_hazard_is_seen():
    mfma = "v_mfma_scale_f32_16x16x128_f8f6f4 v[0:3], a[0:7], a[8:15], 0, v9, v8 op_sel_hi:[0,0,0]"
    assert _hazards(["v_and_b32_e32 v8, 0xff, v8", mfma])[1]
    assert not _hazards(["v_and_b32_e32 v8, 0xff, v8", "s_nop 1", mfma])[1]
    assert _hazards([mfma, "v_add_f32_e32 v4, v1, v4"])[1]
    assert not _hazards([mfma, mfma.replace("v[0:3]", "v[4:7]"), mfma.replace("v[0:3]", "v[10:13]"),
                         "v_add_f32_e32 v20, v1, v20"])[1]


def test_built_code_keeps_its_distances(tmp_path):
    lib = objects.LIBS[0]
    if not os.path.exists(lib):
        pytest.skip("libconvrot.so not built")
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump")
    checked = 0
    for n, (_, code) in enumerate(objects._device_code_objects(open(lib, "rb").read())):
        if not any("fp8_gemm_wide" in k[".name"] for k in objects._kernels(code)):
            continue
        path = tmp_path / f"{n}.co"
        path.write_bytes(code)
        text = subprocess.run([OBJDUMP, "-d", "--mcpu=gfx950", str(path)], capture_output=True, text=True,
                              check=True).stdout
        lines = [ln.split("//")[0].strip() for ln in text.splitlines() if ln.startswith("\t")]
        count, found = _hazards([ln for ln in lines if ln])
        assert not found, found[:5]
        checked += count
    assert checked >= 4 * 128, checked  # four kernels of several half-blocks each
