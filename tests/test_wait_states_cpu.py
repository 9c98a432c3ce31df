"""Wait states in the built library's gfx950 code: no GPU.

gfx9 leaves two to software where a buffer load copies into LDS.  The compiler
inserts them for instructions of its own, but does not look into inline asm:

* one between a scalar write of m0 and the load;
* five between a vector instruction's write of a scalar register and a vector
  memory instruction that reads it.

gfx950 leaves two more between such a write and a vector instruction that reads
the register as a mask, as the carry of an addition that inline asm writes.
"""

import os
import re
import shutil
import subprocess

import pytest

from blockwise_scaled_fp8_bs_amd import _lib

OBJDUMP = os.environ.get("LLVM_OBJDUMP", "/opt/rocm/llvm/bin/llvm-objdump")
SGPR_TO_VMEM, M0_TO_LDS, SGPR_TO_MASK = 5, 1, 2

_RANGE, _ONE = re.compile(r"\bs\[(\d+):(\d+)\]"), re.compile(r"\bs(\d+)\b")


def scalars(text):
    """Scalar registers that operands name."""
    found = {int(n) for n in _ONE.findall(text)}
    for lo, hi in _RANGE.findall(text):
        found.update(range(int(lo), int(hi) + 1))
    return found | ({"vcc"} if "vcc" in text else set())


def vector_writes(op, operands):
    """Scalar registers that a vector instruction writes."""
    if op.startswith(("v_readlane", "v_readfirstlane")) or (op.startswith("v_cmp") and not op.startswith("v_cmpx")):
        return scalars(operands[0])
    return scalars(operands[1]) if op.startswith("v_") and len(operands) > 2 and re.search("_co_|div_scale|mad_[ui]64", op) else set()


def hazards(lines):
    """Copies into LDS in a listing, and those among them, and additions with a carry, that come too early (in the
    listing's order)."""
    loads, early = 0, []
    recent = []  # of the last instructions: states since, scalar registers written by a vector one, m0 written
    for line in lines:
        line = line.split("//")[0].strip()
        if not line or line.endswith(":") or not re.match(r"[a-z]+_", line):
            continue
        op, _, rest = line.partition(" ")
        operands = [o.strip() for o in rest.split(",")]
        if op.startswith("buffer_load") and rest.split()[-1] == "lds":
            loads += 1
            used = scalars(rest)
            if any((age < SGPR_TO_VMEM and used & written) or (age < M0_TO_LDS and m0) for age, written, m0 in recent):
                early.append(line)
        if op == "v_addc_co_u32_e64" and any(age < SGPR_TO_MASK and scalars(operands[4]) & written for age, written, _ in recent):
            early.append(line)
        states = int(rest, 0) + 1 if op == "s_nop" else 1
        recent = [(age + states, written, m0) for age, written, m0 in recent if age + states < SGPR_TO_VMEM]
        recent.append((0, vector_writes(op, operands), op.startswith("s_") and operands[0] == "m0"))
    return loads, early


def test_what_is_looked_for():
    load = "buffer_load_dwordx4 v1, s[4:7], s9 offen lds"
    nop = "s_nop 3"
    assert hazards(["s_mov_b32 m0, s2", load]) == (1, [load])
    assert hazards(["s_mov_b32 m0, s2", "s_nop 0", load]) == (1, [])
    for write in ("v_readlane_b32 s7, v2, 3", "v_readfirstlane_b32 s9, v0", "v_cmp_lt_i32_e64 s[8:9], v0, v1",
                  "v_add_co_u32_e64 v3, s[6:7], v1, v2"):
        assert hazards([write, "s_mov_b32 m0, s2", "s_nop 2", load]) == (1, [load])
        assert hazards([write, "s_mov_b32 m0, s2", nop, load]) == (1, [])
    add = "v_addc_co_u32_e64 v1, s[0:1], v1, v1, s[2:3]"
    assert hazards(["v_cmp_lt_i32_e64 s[2:3], v0, v1", "s_nop 0", add]) == (0, [add])
    assert hazards(["v_cmp_lt_i32_e64 s[2:3], v0, v1", "s_nop 1", add]) == (0, [])
    assert hazards(["v_readfirstlane_b32 s2, v0", "s_mov_b32 m0, s2", "s_nop 0", load, "v_mov_b32_e32 v1, s9"]) == (1, [])


def test_copies_into_lds(tmp_path):
    if not os.path.exists(_lib.LIB_PATH):
        pytest.fail("libbs.so is not built (python -m blockwise_scaled_fp8_bs_amd.build)")
    if not os.path.exists(OBJDUMP):
        pytest.skip("needs llvm-objdump")
    lib = shutil.copy(_lib.LIB_PATH, tmp_path / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", str(lib)], check=True, cwd=tmp_path, stdout=subprocess.DEVNULL)
    total, early = 0, []
    for name in sorted(os.listdir(tmp_path)):
        if "gfx950" not in name:
            continue
        with subprocess.Popen([OBJDUMP, "-d", "--no-show-raw-insn", name], cwd=tmp_path, stdout=subprocess.PIPE, text=True) as p:
            n, e = hazards(p.stdout)
        assert p.returncode == 0
        total += n
        early += e
    assert total > 1000 and not early, (total, len(early), early[:5])
