"""The attention kernels' matrix instructions, which are inline assembly, keep the distances that they
need, in both register files and round the loops (CPU).

As test_matrix_registers.py, for v_mfma_f32_32x32x16_bf16: no vector instruction writes an operand less
than 2 wait states before it, nothing touches its result for 18 wait states, but another of these
instructions onto the same sums may follow at any distance, and nothing writes what it adds to for 11: it
reads that after it has been issued.  Each occupies the matrix core for 8.

Skipped when the library has not been built or there is no disassembler.
"""

import os
import re
import subprocess

import pytest

import test_code_objects as objects
import test_matrix_registers as registers
from test_matrix_hazards import OBJDUMP

MFMA = "v_mfma_f32_32x32x16_bf16"
NAME = re.compile(r"attention_kernelILi")
OPERAND_STATES, RESULT_STATES, ADDEND_STATES, MFMA_STATES = 2, 18, 11, 8


def _hazards(ins):
    found, count = [], 0
    for m in ins:
        if not m.mfma:
            continue
        assert m.op == MFMA, m.op
        count += 1
        open_, seen = [(p, 0) for p in m.before], {}
        while open_:
            p, states = open_.pop()
            if states >= OPERAND_STATES or seen.get(p, OPERAND_STATES) <= states:
                continue
            seen[p] = states
            if p.writes & m.operands:
                found.append(f"{p.text} -> {m.text}")
            open_ += [(q, states + p.states()) for q in p.before]
        open_, seen = [(p, 0) for p in m.after], {}
        while open_:
            p, states = open_.pop()
            if states >= RESULT_STATES or seen.get(p, RESULT_STATES) <= states:
                continue
            seen[p] = states
            onto = p.mfma and p.result == m.result and \
                not registers._registers(",".join(registers._fields(p.text)[1][1:3])) & m.result
            if p.uses & m.result and not onto:
                found.append(f"{m.text} <- {p.text}")
            open_ += [(q, states + (MFMA_STATES if p.mfma else p.states())) for q in p.after]
        addend = registers._registers(registers._fields(m.text)[1][3]) - m.result
        open_, seen = [(p, 0) for p in m.after], {}
        while open_:
            p, states = open_.pop()
            if states >= ADDEND_STATES or seen.get(p, ADDEND_STATES) <= states:
                continue
            seen[p] = states
            if p.writes & addend:
                found.append(f"{m.text} overwritten by {p.text}")
            open_ += [(q, states + (MFMA_STATES if p.mfma else p.states())) for q in p.after]
    return count, found


def test_planted_hazards_are_seen():
    score = MFMA + " v[0:15], v[32:35], a[0:3], v[0:15]"
    other = MFMA + " a[16:31], v[36:39], v[40:43], a[16:31]"

    def seen(*texts):
        return bool(_hazards(registers._straight(*texts))[1])

    assert seen("v_cvt_pk_bf16_f32 v40, v50, v51", other)
    assert not seen("v_cvt_pk_bf16_f32 v40, v50, v51", "s_nop 1", other)
    assert seen(score, "v_fma_f32 v60, v3, v61, v62")
    assert seen(score, other, "v_fma_f32 v60, v3, v61, v62")
    assert not seen(score, other, "s_nop 9", "v_fma_f32 v60, v3, v61, v62")
    assert not seen(score, score) and seen(score, MFMA + " a[16:31], v[0:3], v[40:43], a[16:31]")
    assert seen(other, "v_accvgpr_read_b32 v60, a20")
    first = MFMA + " v[0:15], v[32:35], a[0:3], v[16:31]"
    assert seen(first, "v_add_u32_e32 v30, s74, v115") and seen(first, other, "v_add_u32_e32 v30, s74, v115")
    assert not seen(first, "s_nop 10", "v_add_u32_e32 v30, s74, v115")


def test_built_code_keeps_its_distances(tmp_path):
    lib = objects.LIBS[0]
    if not os.path.exists(lib):
        pytest.skip("libconvrot.so not built")
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump")
    kernels = {}
    for n, (_, code) in enumerate(objects._device_code_objects(open(lib, "rb").read())):
        if not any("attention_kernel" in k[".name"] for k in objects._kernels(code)):
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
            elif ln.startswith("\t") and "//" in ln:
                ins, _, note = ln.partition("//")
                address = int(re.match(r"\s*([0-9A-F]+):", note)[1], 16)
                target = re.search(r"<[^>+]+(?:\+0x([0-9a-f]+))?>\s*$", note)
                branch = ins.strip().startswith(("s_branch", "s_cbranch"))
                assert branch == bool(target), ln
                kernels[name].append((address, ins.strip(), start + int(target[1] or "0", 16) if branch else None))
    kernels = {name: registers._kernel(lines) for name, lines in kernels.items() if NAME.search(name)}
    assert len(kernels) == 20  # for 5 sizes of heads, with and without a mask, few and many queries
    for name, ins in kernels.items():
        count, found = _hazards(ins)
        assert count >= 16, (name, count)
        assert not found, (name, len(found), found[:8])
