"""Wait states of the direct-to-LDS loads in the built library's machine code.

These loads stand in inline assembly, where the compiler adds no wait states, and
take the LDS address from m0 and the buffer from scalar registers.  gfx950 wants
one wait state between a scalar write of m0 and such a load, and five between a
vector instruction's write of a scalar register and a memory instruction that
reads it; too few are no error, the load then takes the registers' old values."""
import os
import re
import shutil
import subprocess

import pytest

from moe_grouped_gemm_bf16_amd import _lib

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
MEMORY = ("buffer_", "global_", "scratch_", "flat_")
NO_RESULT = ("s_cmp", "s_bitcmp", "s_nop", "s_wait", "s_branch", "s_cbranch", "v_nop", "v_cmpx")


def _scalars(token):
    """The scalar registers that an operand names."""
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", token)
    if m:
        return {f"s{i}" for i in range(int(m[1]), int(m[2]) + 1)}
    if token == "vcc":
        return {"vcc_lo", "vcc_hi"}
    return {token} if re.fullmatch(r"s\d+|m0|vcc_lo|vcc_hi", token) else set()


def _hazards(lines):
    """(direct-to-LDS loads, hazards) of a disassembly."""
    loads, found, name, before = 0, [], "", []          # before: (op, states, scalars written)
    for line in lines:
        m = re.match(r"^[0-9a-f]+ <(.*)>:", line)
        if m:
            name, before = m[1], []
            continue
        op, _, rest = line.split("//")[0].strip().partition(" ")
        if not op:
            continue
        tokens = [t for part in re.split(r",(?![^\[]*\])", rest) for t in part.split()]
        if op.startswith(MEMORY):
            lds = "lds" in tokens
            loads += lds
            read = set().union(*map(_scalars, tokens)) if tokens else set()
            states = 0
            for o, n, wrote in reversed(before):
                if states < 5 and o.startswith("v_") and wrote & read:
                    found.append((name, o, op, states))
                if states < 1 and lds and o.startswith("s_") and "m0" in wrote:
                    found.append((name, o, op, states))
                states += n
        wrote = set()
        if tokens and op.startswith(("s_", "v_")) and not op.startswith(NO_RESULT):
            # (the second operand: a carry out)
            wrote = _scalars(tokens[0]) | (_scalars(tokens[1]) if "_co_" in op or "div_scale" in op else set())
        before = before[-7:] + [(op, int(tokens[0], 0) + 1 if op == "s_nop" else 1, wrote)]
    return loads, found


def test_the_check_sees_both():
    good = ["0 <k>:", " s_mov_b32 m0, s4", " s_nop 0", " buffer_load_dwordx4 v1, s[8:11], 0 offen lds"]
    assert _hazards(good) == (1, [])
    assert len(_hazards(good[:2] + good[3:])[1]) == 1
    assert len(_hazards(["0 <k>:", " v_readfirstlane_b32 s9, v2", " s_nop 3"] + good[3:])[1]) == 1
    assert _hazards(["0 <k>:", " v_readfirstlane_b32 s9, v2", " s_nop 4"] + good[3:]) == (1, [])
    assert len(_hazards(["0 <k>:", " v_cmp_lt_i32_e64 s[10:11], v0, v1"] + good[3:])[1]) == 1


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="needs llvm-objdump")
def test_no_load_reads_a_register_too_early(tmp_path):
    shutil.copy(_lib.LIB_PATH, tmp_path / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", "lib.so"], cwd=tmp_path, check=True, capture_output=True)
    loads, found = 0, []
    for f in sorted(tmp_path.glob("lib.so.*gfx950")):
        out = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", str(f)], check=True, capture_output=True, text=True)
        n, bad = _hazards(out.stdout.splitlines())
        loads += n
        found += bad
    assert loads > 500                   # the products' loads are there to be seen
    assert not found, (len(found), found[:3])
