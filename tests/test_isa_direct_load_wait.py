"""The machine code of the direct global->LDS loads (no GPU needed).

A load to LDS takes its LDS address from M0.  Between a scalar instruction that
writes M0 and such a load this target needs one wait state: an instruction in
between, s_nop if there is no other.  The compiler keeps to that by itself, but does
not look inside inline assembly, where the loads are written.  The assembled code is
read here, not the compiler's text: what the two look like may differ.
"""
import os
import re
import subprocess

import pytest

from mixture_experts_layer_up_amd import build

SOURCES = [f for f in build.sources()
           if re.search(r'#include "(lds_dma|block_dma)\.h"', open(f).read())]
OBJDUMP = os.path.join(os.path.dirname(os.path.realpath(build.HIPCC)), "..", "lib", "llvm", "bin", "llvm-objdump")
if not os.path.exists(OBJDUMP):
    OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"


def _machine_code(src, tmp_path):
    """Instructions of the device code, in order."""
    out = tmp_path / (os.path.basename(src) + ".o")
    subprocess.run([build.HIPCC, *build.COMMON_FLAGS, "--cuda-device-only", "--no-gpu-bundle-output", "-c", src, "-o",
                    str(out)], check=True, capture_output=True)
    text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", str(out)], check=True, capture_output=True,
                          text=True).stdout
    lines = [ln.split("//")[0].strip() for ln in text.splitlines()]
    return [ln for ln in lines if re.match(r"^[a-z]\w+( |$)", ln)]


def _unwaited(lines):
    """(loads to LDS that directly follow a write of M0, all loads to LDS)."""
    bad, loads = [], 0
    for before, t in zip([""] + lines, lines):
        if re.search(r"^(buffer|global)_load\w*_lds|^(buffer|global|scratch)_load.* lds$", t):
            loads += 1
            if re.match(r"^s_\w+ m0\b", before):
                bad.append((before, t))
    return bad, loads


@pytest.mark.parametrize("src", SOURCES, ids=os.path.basename)
def test_a_wait_state_after_every_write_of_m0(src, tmp_path):
    bad, loads = _unwaited(_machine_code(src, tmp_path))
    assert loads > 0
    assert not bad, f"{len(bad)} of {loads} loads follow the write of M0 at once: {bad[:2]}"


def test_the_check_itself():
    load = ["global_load_lds_dwordx4 v[2:3], off nt", "buffer_load_dwordx4 v4, s[8:11], 0 offen lds"]
    for t in load:
        assert _unwaited(["s_mov_b32 m0, s4", t]) == ([("s_mov_b32 m0, s4", t)], 1)
        assert _unwaited(["s_add_u32 m0, s4, 64", t])[0]
        assert _unwaited(["s_mov_b32 m0, s4", "s_nop 0", t]) == ([], 1)
        assert _unwaited(["s_mov_b32 s4, m0", t]) == ([], 1)
    assert _unwaited(["s_mov_b32 m0, s4", "buffer_load_dwordx4 v[4:7], v1, s[8:11], 0 offen"]) == ([], 0)
