"""The matrix instructions of the cross entropy kernels are written in assembly, so the
compiler does not keep the distances that they need.  This reads the built library's own
code and checks them, for whatever compiler built it:

  - no vector instruction writes an operand in the two wait states before its use;
  - nothing but another matrix instruction touches a result in the 19 wait states after
    it (the most that any of these instructions asks for).

An instruction is one wait state, s_nop n is n + 1.  Both ways out of a branch are
followed."""
from __future__ import annotations

import os
import re
import shutil
import subprocess

import pytest

import sparse_linear_layers_02_amd as sbn

OPERAND, RESULT = 2, 19


def registers(text):
    """The vector registers, of both files, that an operand list names."""
    out = set()
    for f, a, lo, hi in re.findall(r"\b([va])(?:(\d+)\b|\[(\d+):(\d+)\])", text):
        out.update((f, r) for r in (range(int(lo), int(hi) + 1) if lo else (int(a),)))
    return out


def parse(lines):
    """[(address, mnemonic, [operands], address branched to or None)] of one function's listing."""
    out, start = [], None
    for line in lines:
        m = re.match(r"\s*([a-z]\w+)\s*(.*?)\s*//\s*([0-9A-F]+):[0-9A-F ]*(?:<[^>]*\+0x([0-9a-f]+)>|<[^>+]*>)?\s*$", line)
        if not m:
            continue
        at = int(m[3], 16)
        start = at if start is None else start
        operands = re.split(r",\s*(?![^\[]*\])", m[2]) if m[2] else []
        to = start + int(m[4] or "0", 16) if "branch" in m[1] else None
        out.append((at, m[1], operands, to))
    return out


def hazards(code):
    """Descriptions of every distance that is too short."""
    place = {at: i for i, (at, *_) in enumerate(code)}
    found = set()

    def walk(i, need, left, skip, wrong):
        """From instruction i on for `left` wait states, over all ways that the code may take."""
        work = [(i, left)]
        seen = {}
        while work:
            i, left = work.pop()
            if left <= 0 or i >= len(code) or seen.get(i, 0) >= left:
                continue
            seen[i] = left
            at, op, operands, to = code[i]
            if wrong(op, operands, need) and not skip(op):
                found.add(f"{at:x}: {op} {', '.join(operands)} ({left} wait states early)")
            left -= int(operands[0], 0) + 1 if op == "s_nop" else 1
            if to is not None:
                work.append((place[to], left))
            if op not in ("s_branch", "s_endpgm"):
                work.append((i + 1, left))

    mfma = lambda op: op.startswith("v_mfma")  # noqa: E731
    touches = lambda op, operands, need: any(registers(x) & need for x in operands)  # noqa: E731
    uses = lambda op, operands, need: mfma(op) and any(registers(x) & need for x in operands[1:])  # noqa: E731
    for i, (at, op, operands, to) in enumerate(code):
        if mfma(op):
            walk(i + 1, registers(operands[0]), RESULT, mfma, touches)
        elif op.startswith("v_") and operands and not op.startswith(("v_cmp", "v_readfirstlane", "v_readlane", "v_nop")):
            wrote = registers(operands[0]) | (registers(operands[1]) if "swap" in op else set())
            if wrote:
                walk(i + 1, wrote, OPERAND, lambda op: False, uses)
    return found


def listing(*instructions):
    return parse([f"\t{x.split(' <')[0]} // {16 * i:012X}: 00000000 {'<' + x.split(' <')[1] if ' <' in x else ''}"
                  for i, x in enumerate(instructions)])


@pytest.mark.parametrize("bad,code", [
    (0, ["v_mov_b32_e32 v4, v9", "s_nop 1", "v_mfma_f32_16x16x32_bf16 a[0:3], v[4:7], v[0:3], a[0:3]", "s_nop 15", "s_nop 2",
         "v_accvgpr_read_b32 v1, a2"]),
    (1, ["v_mov_b32_e32 v4, v9", "s_nop 0", "v_mfma_f32_16x16x32_bf16 a[0:3], v[4:7], v[0:3], a[0:3]"]),
    (1, ["v_accvgpr_write_b32 a3, 0", "v_mfma_f32_16x16x32_bf16 a[0:3], v[4:7], v[0:3], a[0:3]"]),
    (1, ["v_permlane16_swap_b32_e32 v9, v5", "v_mfma_f32_16x16x32_bf16 a[0:3], v[4:7], v[0:3], a[0:3]"]),
    (1, ["v_mfma_f32_16x16x32_bf16 a[0:3], v[4:7], v[0:3], a[0:3]", "s_nop 15", "s_nop 1", "v_accvgpr_read_b32 v1, a2"]),
    (1, ["v_mfma_f32_16x16x32_bf16 a[0:3], v[4:7], v[0:3], a[0:3]", "v_accvgpr_write_b32 a0, 0"]),
    (0, ["v_mfma_f32_16x16x32_bf16 a[0:3], v[4:7], v[0:3], a[0:3]", "v_mfma_f32_16x16x32_bf16 a[0:3], v[4:7], v[0:3], a[0:3]"]),
    # around a loop: the next round's first instruction reads the last one's result
    (1, ["v_accvgpr_read_b32 v1, a2", "s_nop 7", "v_mfma_f32_16x16x32_bf16 a[0:3], v[4:7], v[0:3], a[0:3]",
         "s_cbranch_scc1 65530 <f+0x0>", "s_endpgm"]),
])
def test_the_check_itself(bad, code):
    assert len(hazards(listing(*code))) == bad


def test_matrix_instructions_keep_their_distances(tmp_path):
    tools = "/opt/rocm/llvm/bin"
    if not os.path.exists(os.path.join(tools, "llvm-objdump")):
        pytest.skip("no disassembler for gfx950")
    lib = shutil.copy(sbn.LIB_PATH, tmp_path)
    dump = os.path.join(tools, "llvm-objdump")
    subprocess.run([dump, "--offloading", lib], check=True, cwd=tmp_path, capture_output=True)
    kernels = products = 0
    for f in sorted(os.listdir(tmp_path)):
        if not f.endswith("gfx950"):
            continue
        text = subprocess.run([dump, "-d", "--mcpu=gfx950", f], check=True, cwd=tmp_path, capture_output=True, text=True).stdout
        for body in re.split(r"^[0-9a-f]+ <", text, flags=re.M)[1:]:
            name, _, body = body.partition(">:")
            if "ce_gemm_kernel" not in name:
                continue
            code = parse(body.splitlines())
            assert code[-1][0] - code[0][0] > 1000 and any(to is not None for *_, to in code), name
            kernels += 1
            products += sum(op.startswith("v_mfma") for _, op, *_ in code)
            assert not hazards(code), name
    assert kernels >= 18 and products > 1000
