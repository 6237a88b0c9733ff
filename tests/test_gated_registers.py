"""The gated pair's wide kernels keep the distances that their matrix instructions, written as inline
assembly, need: the checks of test_matrix_registers.py on the built code of fp8_gated.hip (CPU).

Skipped when the library has not been built or there is no disassembler.
"""

import os
import re
import subprocess

import pytest

import test_code_objects as objects
from test_matrix_hazards import OBJDUMP
from test_matrix_registers import _hazards, _kernel

NAME = "fp8_gated_wide"


def test_built_code_keeps_its_distances(tmp_path):
    lib = objects.LIBS[0]
    if not os.path.exists(lib):
        pytest.skip("libconvrot.so not built")
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump")
    kernels = {}
    for n, (_, code) in enumerate(objects._device_code_objects(open(lib, "rb").read())):
        if not any(NAME in k[".name"] for k in objects._kernels(code)):
            continue
        path = tmp_path / f"{n}.co"
        path.write_bytes(code)
        text = subprocess.run([OBJDUMP, "-d", "--mcpu=gfx950", str(path)], capture_output=True, text=True,
                              check=True).stdout
        name = start = None
        for ln in text.splitlines():
            head = re.match(r"([0-9a-f]+) <(.+)>:$", ln)
            if head:
                start, name = int(head[1], 16), head[2]
                kernels[name] = []
            elif ln.startswith("\t") and "//" in ln and NAME in name:
                ins, _, note = ln.partition("//")
                address = int(re.match(r"\s*([0-9A-F]+):", note)[1], 16)
                target = re.search(r"<[^>+]+(?:\+0x([0-9a-f]+))?>\s*$", note)
                branch = ins.strip().startswith(("s_branch", "s_cbranch"))
                assert branch == bool(target), ln
                kernels[name].append((address, ins.strip(), start + int(target[1] or "0", 16) if branch else None))
    kernels = {name: _kernel(lines) for name, lines in kernels.items() if NAME in name}
    assert len(kernels) == 4  # both kinds of weight scales, with and without kept projections
    for name, ins in kernels.items():
        count, found = _hazards(ins)
        assert count >= 128, (name, count)
        assert not found, (name, len(found), found[:8])
