"""Wait states before the LDS DMA loads (no GPU): the compiler inserts none for inline asm, so the
helpers of csrc/dma.hpp and the attention kernels carry their own.  The library's gfx950 code is
disassembled and every load into LDS is checked against what the gfx9 ISA asks for:

  * one wait state between a write of M0, which holds the LDS address, and the load;
  * five between a vector instruction's write of a scalar register (readfirstlane, readlane, a
    comparison's mask) and a load that takes the register in its buffer descriptor.

An instruction in between is one wait state, s_nop N is N + 1."""

import os
import re
import shutil
import subprocess

import pytest

from fp8_quantized_gemm_amax_amd import LIB_PATH

OBJDUMP = next((p for p in (shutil.which("llvm-objdump"), "/opt/rocm/llvm/bin/llvm-objdump") if p and os.path.exists(p)), None)
DMA = re.compile(r"^(buffer_load_\w+ .*\blds$|global_load_lds_\w+ )")
REGS = re.compile(r"\b([sv])(?:\[(\d+):(\d+)\]|(\d+)\b)|\bm0\b")


def scalars(text):
    """Scalar registers named in an operand text: numbers, and 'm0'."""
    found = set()
    for m in REGS.finditer(text):
        if m.group(0) == "m0":
            found.add("m0")
        elif m.group(1) == "s":
            lo = int(m.group(2) or m.group(4))
            found.update(range(lo, int(m.group(3) or lo) + 1))
    return found


def writes(line):
    """(scalar registers written, by a vector instruction?) of one instruction."""
    name, _, rest = line.partition(" ")
    if name[:2] not in ("s_", "v_") or name.startswith(("s_cmp", "s_bitcmp", "s_waitcnt", "s_nop", "s_cbranch", "s_setprio")):
        return set(), False
    operands = re.split(r",\s*", rest)
    if name.startswith("v_"):     # destinations: the first operand, and the carry or the mask after a vector one
        first = scalars(operands[0])
        if not first and re.match(r"v_(add|sub|subrev|addc|subb|subbrev)_co_|v_div_scale|v_mad_[iu]64", name):
            first = scalars(operands[1])
        return first, True
    return scalars(operands[0]), False


def states(line):
    m = re.match(r"s_nop (\d+)", line)
    return int(m.group(1)) + 1 if m else 1


def problems(lines):
    """(LDS DMA loads found, those with too few wait states) in a list of instructions."""
    count, bad = 0, []
    for i, line in enumerate(lines):
        if not DMA.match(line):
            continue
        count += 1
        reads = {"m0"} | scalars(line)
        passed = 0
        for j in range(i - 1, -1, -1):
            before = lines[j]
            if passed >= 5 or before.startswith(("s_branch", "s_endpgm", "s_setpc")):
                break
            regs, vector = writes(before)
            need = 5 if vector else 1
            hit = regs & (reads if vector else {"m0"})
            if hit and passed < need:
                bad.append(f"{before}  ->  {line}  ({passed} of {need} wait states)")
            passed += states(before)
    return count, bad


def disassembled(folder):
    """The library's gfx950 instructions, one list per code object."""
    copy = os.path.join(folder, "lib.so")
    shutil.copy(LIB_PATH, copy)
    subprocess.run([OBJDUMP, "--offloading", "lib.so"], cwd=folder, check=True, capture_output=True, timeout=300)
    for name in sorted(os.listdir(folder)):
        if name.endswith("gfx950"):
            r = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", name], cwd=folder, check=True, capture_output=True, text=True, timeout=300)
            yield [x.split("//")[0].strip() for x in r.stdout.splitlines() if x.startswith("\t")]


def test_the_check_itself():
    dma = "buffer_load_dwordx4 v21, s[4:7], 0 offen lds"
    assert problems(["s_mov_b32 m0, 0", dma]) == (1, [f"s_mov_b32 m0, 0  ->  {dma}  (0 of 1 wait states)"])
    assert problems(["s_cselect_b32 m0, 0x400, -1", "s_nop 0", dma]) == (1, [])
    assert problems(["s_mov_b32 m0, s3", "v_add_u32_e32 v1, v2, v3", dma]) == (1, [])
    assert len(problems(["v_readfirstlane_b32 s6, v1", "s_mov_b32 m0, 0", "s_nop 2", dma])[1]) == 1
    assert problems(["v_readfirstlane_b32 s6, v1", "s_nop 3", "s_mov_b32 m0, 0", "s_nop 0", dma]) == (1, [])
    assert problems(["v_readfirstlane_b32 s8, v1", "s_mov_b32 m0, 0", "s_nop 0", dma]) == (1, [])
    assert len(problems(["v_readfirstlane_b32 m0, v1", "s_nop 0", "global_load_lds_dword v[4:5], off"])[1]) == 1
    assert problems(["v_cmp_lt_i32_e64 s[2:3], v1, v2", "s_nop 0", "s_mov_b32 m0, 1", "s_branch 12", dma]) == (1, [])


def test_lds_dma_has_its_wait_states(tmp_path):
    if OBJDUMP is None or not os.path.exists(LIB_PATH):
        pytest.skip("no llvm-objdump, or the library has not been built")
    total, bad = 0, []
    for lines in disassembled(str(tmp_path)):
        n, b = problems(lines)
        total += n
        bad += b
    assert total > 3000, total
    assert not bad, f"{len(bad)} of {total} LDS DMA loads: {bad[:3]}"
