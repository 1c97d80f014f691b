"""The instructions of the built kernels, where a rule of the hardware lies with the source and not
with the compiler, which does not look into asm."""
import glob
import os
import re
import shutil
import subprocess

import pytest

import mxfp4_expert_gemm_amd as moe

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"

pytestmark = [pytest.mark.skipif(not os.path.exists(moe.LIB_PATH), reason="libmoe_layer.so not built"),
              pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="needs llvm-objdump")]


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """(kernel, its instructions) of the library's device code."""
    d = tmp_path_factory.mktemp("listing")
    shutil.copy(moe.LIB_PATH, d / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", "lib.so"], cwd=d, check=True, capture_output=True)
    found = []
    for obj in sorted(glob.glob(str(d / "lib.so.*gfx950"))):
        name, lines = None, []
        p = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", "--no-leading-addr", obj], capture_output=True, text=True,
                           check=True)
        for line in p.stdout.splitlines():
            m = re.match(r"^(?:[0-9a-f]+ )?<(\S+)>:$", line)
            if m:
                name, lines = m.group(1), []
                found.append((name, lines))
            elif name and line.strip():
                lines.append(line.split("//")[0].strip())
    return found


def lds_loads_behind_m0(lines):
    """(loads into LDS, those of them right behind the write of m0 that they read)"""
    loads = [i for i, s in enumerate(lines) if re.match(r"(global_load_lds|buffer_load\S* .*\blds\b)", s)]
    return len(loads), [i for i in loads if i and re.match(r"s_\S+ m0,", lines[i - 1])]


def test_the_search_sees_a_missing_wait():
    lines = ["s_mov_b32 m0, s4", "s_nop 0", "global_load_lds_dwordx4 v[0:1], off", "s_add_u32 m0, s4, s5",
             "global_load_lds_dwordx4 v2, s[2:3]"]
    assert lds_loads_behind_m0(lines) == (2, [4])


def test_a_load_into_lds_waits_for_m0(kernels):
    """One wait state lies between a write of m0 and a load into LDS, which takes its place from there."""
    total = 0
    for name, lines in kernels:
        n, bad = lds_loads_behind_m0(lines)
        total += n
        assert not bad, f"{name}: {len(bad)} of {n} loads, first at instruction {bad[0]}"
    assert total > 1000  # the listing was read
