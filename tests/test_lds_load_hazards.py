"""Loads from memory into LDS take their LDS address from M0, and those of this
library stand in inline assembly, where the compiler looks after no hazard: one
wait state has to pass between a scalar write of M0 and such a load, and five
between a vector instruction's write of a scalar register and a load whose base
address it holds.  Looked up in the disassembly of the built library."""
import os
import re
import shutil
import subprocess

import pytest

import quantized_linear_layer_amd as qll

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"


def scalar_registers(text):
    regs = {int(r) for r in re.findall(r"\bs(\d+)\b", text)}
    for lo, hi in re.findall(r"\bs\[(\d+):(\d+)\]", text):
        regs |= set(range(int(lo), int(hi) + 1))
    return regs


def hazards(lines):
    """(loads into LDS, faults) of a disassembly: instructions in program order."""
    loads, faults, before = 0, [], []
    for line in lines:
        line = line.split("//")[0].strip()
        if line.endswith(">:"):  # a new kernel
            before = []
            continue
        if not line or line.endswith(":"):
            continue
        op, _, rest = line.partition(" ")
        if re.match(r"(global|buffer|scratch)_load_lds_|buffer_load_.* lds$", line):
            loads += 1
            states, base = 0, scalar_registers(rest)
            for was, args in reversed(before[-6:]):
                if states < 1 and was.startswith("s_") and re.match(r"m0\b", args):
                    faults.append((was + " " + args, line))
                if states < 5 and was.startswith("v_") and scalar_registers(args.split(",")[0]) & base:
                    faults.append((was + " " + args, line))
                states += 1 + (int(args, 0) if was == "s_nop" else 0)
        before.append((op, rest.strip()))
    return loads, faults


@pytest.mark.parametrize("lines,count", [
    (["s_mov_b32 m0, s4", "global_load_lds_dwordx4 v0, s[2:3]"], 1),
    (["s_mov_b32 m0, s4", "s_nop 0", "global_load_lds_dwordx4 v0, s[2:3]"], 0),
    (["s_add_u32 m0, s4, 16", "buffer_load_dword v1, s[4:7], 0 offen lds"], 1),
    (["v_readfirstlane_b32 s3, v9", "s_mov_b32 m0, s4", "s_nop 0", "global_load_lds_ushort v0, s[2:3]"], 1),
    (["v_readfirstlane_b32 s3, v9", "s_mov_b32 m0, s4", "s_nop 3", "global_load_lds_ushort v0, s[2:3]"], 0),
    (["v_readfirstlane_b32 s5, v9", "s_mov_b32 m0, s4", "s_nop 0", "global_load_lds_ushort v0, s[2:3]"], 0)])
def test_what_counts_as_a_hazard(lines, count):
    loads, faults = hazards(lines)
    assert loads == 1 and len(faults) == count


def test_loads_into_lds_wait_for_their_address(tmp_path):
    if not os.path.exists(OBJDUMP):
        pytest.skip("no disassembler")
    lib = tmp_path / "lib.so"
    shutil.copy(qll.LIB_PATH, lib)
    subprocess.run([OBJDUMP, "--offloading", "lib.so"], cwd=tmp_path, check=True, capture_output=True)
    objects = sorted(tmp_path.glob("lib.so.*gfx950*"))
    assert objects
    loads, faults = 0, []
    for obj in objects:
        out = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", str(obj)], check=True, capture_output=True,
                             text=True).stdout
        n, bad = hazards(out.splitlines())
        loads, faults = loads + n, faults + bad
    assert loads > 0
    assert not faults, f"{len(faults)} of {loads} loads, the first: {faults[0]}"
