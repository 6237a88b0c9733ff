"""Matrix instructions written as inline assembly keep their distances in both register files and
round every loop (CPU).

The built gfx950 code of fp8_gemm_wide.hip is disassembled into the graph of its instructions, and
for every v_mfma_scale of its kernels, whether its registers are vector (v) or accumulation (a) ones:

* no vector instruction (a copy into an accumulation register is one) writes an operand less than 2
  wait states before it, on any path that leads there;
* nothing but a wait touches its result for 18 wait states, on any path that leads on.  Another matrix
  instruction of this size occupies the matrix core, and with it the issue of the next one, for 8.

Skipped when the library has not been built or there is no disassembler.
"""

import os
import re
import subprocess

import pytest

import test_code_objects as objects
from test_matrix_hazards import OBJDUMP

MFMA = "v_mfma_scale_f32_16x16x128_f8f6f4"
OPERAND_STATES, RESULT_STATES, MFMA_STATES = 2, 18, 8


def _registers(text):
    """{("v" or "a", number)} of an instruction's text."""
    out = set()
    for f, lo, hi, g, one in re.findall(r"\b([va])\[(\d+):(\d+)\]|\b([va])(\d+)\b", text):
        out |= {(g, int(one))} if g else {(f, r) for r in range(int(lo), int(hi) + 1)}
    return out


def _fields(ins):
    """(opcode, operand texts): commas inside brackets do not separate."""
    op, _, rest = ins.partition(" ")
    return op, [t.strip() for t in re.split(r",(?![^\[]*\])", rest)] if rest else []


class Instruction:
    def __init__(self, text):
        self.text = text
        self.op, fields = _fields(text)
        self.mfma = self.op.startswith("v_mfma")
        self.uses = _registers(" ".join(fields))
        vector = self.op.startswith("v_") and not self.mfma and not self.op.startswith("v_cmp")
        both = "swap" in self.op  # both operands are written
        self.writes = _registers(" ".join(fields[:2 if both else 1])) if vector else set()
        self.result = _registers(fields[0]) if self.mfma else set()
        self.operands = _registers(" ".join(fields[1:])) if self.mfma else set()
        self.before, self.after = [], []

    def states(self):
        return 1 + int(self.text.split()[1], 0) if self.op == "s_nop" else 1


def _kernel(lines):
    """Instructions of one kernel, linked; lines are (address, text, branch target or None)."""
    ins = [Instruction(text) for _, text, _ in lines]
    at = {address: i for i, (address, _, _) in enumerate(lines)}
    for i, (_, _, target) in enumerate(lines):
        assert not ins[i].op.startswith(("s_setpc", "s_swappc", "s_call", "s_cbranch_g"))
        ends = ins[i].op in ("s_endpgm", "s_branch")
        follow = ([] if ends or i + 1 == len(ins) else [i + 1]) + ([] if target is None else [at[target]])
        for j in follow:
            ins[i].after.append(ins[j])
            ins[j].before.append(ins[i])
    return ins


def _hazards(ins):
    """(matrix instructions looked at, descriptions of what comes too early)."""
    found, count = [], 0
    for m in ins:
        if not m.op.startswith("v_mfma_scale"):
            continue
        assert m.op == MFMA, m.op  # (the states above are this one's)
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
            if p.uses & m.result:
                found.append(f"{m.text} <- {p.text}")
            open_ += [(q, states + (MFMA_STATES if p.mfma else p.states())) for q in p.after]
    return count, found


def _straight(*texts):
    return _kernel([(4 * i, t, None) for i, t in enumerate(texts)])


def test_planted_hazards_are_seen():
    one = MFMA + " v[0:3], a[0:7], a[8:15], 0, v9, v8 op_sel_hi:[0,0,0]"
    onto = MFMA + " a[0:3], v[16:23], v[24:31], a[0:3], v9, v8 op_sel_hi:[0,0,0]"
    other = [MFMA + f" v[{r}:{r + 3}], a[16:23], a[24:31], 0, v9, v8 op_sel_hi:[0,0,0]" for r in (40, 44)]
    other_a = [t.replace("v[40:43]", "a[40:43]").replace("v[44:47]", "a[44:47]") for t in other]

    def seen(*texts):
        return bool(_hazards(_straight(*texts))[1])

    # operands, in either file
    assert seen("v_accvgpr_write_b32 a7, v100", one)
    assert seen("v_accvgpr_write_b32 a7, v100", "s_nop 0", one)
    assert not seen("v_accvgpr_write_b32 a7, v100", "s_nop 1", one)
    assert not seen("v_accvgpr_write_b32 a32, v100", one)
    assert seen("v_and_b32_e32 v8, 0xff, v8", "v_mov_b32_e32 v50, v51", one)
    assert seen("v_permlane32_swap_b32_e32 v60, v20", onto)
    assert seen("v_add_f32_e32 v24, v1, v2", onto)
    # results, in either file
    assert seen(one, "v_add_f32_e32 v60, v1, v61")
    assert seen(onto, "v_accvgpr_read_b32 v60, a3")
    assert seen(onto, other_a[0], other_a[1], "v_accvgpr_read_b32 v60, a3")
    assert not seen(onto, other_a[0], other_a[1], "s_nop 1", "v_accvgpr_read_b32 v60, a3")
    assert not seen(onto, "s_nop 15", "s_nop 3", "v_accvgpr_read_b32 v60, a3")
    assert seen(onto, "s_nop 15", "v_accvgpr_read_b32 v60, a3")
    assert seen(onto, onto)


def test_planted_hazards_of_loops_are_seen():
    one = MFMA + " v[0:3], a[0:7], a[8:15], 0, v9, v8 op_sel_hi:[0,0,0]"
    loop = [(0, one, None), (4, "s_nop 15", None), (8, "s_nop 3", None),
            (12, "v_accvgpr_write_b32 a7, v100", None), (16, "s_cbranch_scc1 65531", 0), (20, "s_endpgm", None)]
    assert _hazards(_kernel(loop))[1] == ["v_accvgpr_write_b32 a7, v100 -> " + one]
    loop[3] = (12, "v_mov_b32_e32 v100, v101", None)
    assert not _hazards(_kernel(loop))[1]
    out = [(0, "v_mov_b32_e32 v50, v3", None), (4, "s_nop 15", None), (8, "s_nop 3", None), (12, one, None),
           (16, "s_cbranch_scc1 65531", 0), (20, "s_endpgm", None)]
    assert _hazards(_kernel(out))[1] == [one + " <- v_mov_b32_e32 v50, v3"]


def _wide_kernels(tmp_path):
    """{name: instructions} of the built wide kernels."""
    lib = objects.LIBS[0]
    if not os.path.exists(lib):
        pytest.skip("libconvrot.so not built")
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump")
    kernels = {}
    for n, (_, code) in enumerate(objects._device_code_objects(open(lib, "rb").read())):
        if not any("fp8_gemm_wide" in k[".name"] for k in objects._kernels(code)):
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
            elif ln.startswith("\t") and "//" in ln:  # (others are padding between kernels)
                ins, _, note = ln.partition("//")
                address = int(re.match(r"\s*([0-9A-F]+):", note)[1], 16)
                target = re.search(r"<[^>+]+(?:\+0x([0-9a-f]+))?>\s*$", note)
                branch = ins.strip().startswith(("s_branch", "s_cbranch"))
                assert branch == bool(target), ln
                kernels[name].append((address, ins.strip(), start + int(target[1] or "0", 16) if branch else None))
    return {name: _kernel(lines) for name, lines in kernels.items() if "fp8_gemm_wide" in name}


def test_built_code_keeps_its_distances_in_both_register_files(tmp_path):
    kernels = _wide_kernels(tmp_path)
    assert len(kernels) == 4  # with and without GELU, of both kinds of weight scales
    for name, ins in kernels.items():
        count, found = _hazards(ins)
        assert count >= 128, (name, count)  # several half-blocks
        assert any(i.op.startswith("s_cbranch") for i in ins)
        assert not found, (name, len(found), found[:8])
