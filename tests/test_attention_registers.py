"""The built attention kernels use m0 for their direct-to-LDS loads only (CPU).

Those loads are inline assembly that sets m0 without the compiler's knowledge, so nothing that the
compiler generates may depend on it.  Skipped when the library has not been built or there is no
disassembler.
"""

import os
import subprocess

import pytest

import test_code_objects as objects
from test_matrix_hazards import OBJDUMP


def test_m0_is_the_loads_own(tmp_path):
    lib = objects.LIBS[0]
    if not os.path.exists(lib):
        pytest.skip("libconvrot.so not built")
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump")
    loads = 0
    for n, (_, code) in enumerate(objects._device_code_objects(open(lib, "rb").read())):
        if not any("attention_kernel" in k[".name"] for k in objects._kernels(code)):
            continue
        path = tmp_path / f"{n}.co"
        path.write_bytes(code)
        text = subprocess.run([OBJDUMP, "-d", "--mcpu=gfx950", str(path)], capture_output=True, text=True,
                              check=True).stdout
        lines = [ln.split("//")[0].strip() for ln in text.splitlines() if ln.startswith("\t")]
        for a, b, c in zip(lines, lines[1:], lines[2:]):
            if "m0" in a:
                assert a.startswith("s_mov_b32 m0, "), a
                assert b == "s_nop 0" and c.startswith("buffer_load_dwordx4") and c.endswith("lds"), (a, b, c)
                loads += 1
        assert not any(ins.startswith(("s_movrel", "v_movrel", "s_set_gpr_idx")) for ins in lines)
        assert sum(ln.endswith(" lds") for ln in lines) == sum("m0" in ln for ln in lines)
    assert loads > 0
