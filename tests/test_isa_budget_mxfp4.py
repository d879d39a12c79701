"""Instruction budget of the MXFP4 product's main loops (CPU only: hipcc compiles the kernels to gfx950 assembly;
nothing runs on a GPU).

The three kernels load straight into LDS from inline asm, outside the compiler's wait tracking, and wait for
counts of loads.  These checks pin every loop that holds matrix instructions: its instructions, no spill traffic
and no other memory access in it (a wait by count would then wait for something else), the loads that the counts
stand for, no wait for every access in flight; and the scratch memory of each kernel."""
import re
import subprocess

import pytest

from group_gemm_amd import build as B
from test_isa_budget import innermost_loops

# kernel: (mangled-name prefix of every instantiation, how many, {matrix instructions of a loop: most instructions},
#          loads of a panel in the loop, the count that the loop waits for, most scratch bytes per lane).  The tile
#          kernel's loops hold its 16 loads and both forms of the scales' (one load, or four of 4 bytes): the counts
#          stand for the fewer.  Its 512 registers are all in use: some values around the loops are spilled.
KERNELS = {
    "stream": ("_ZN2gg3fp46stream6kernel", 6, {2: 98}, 3, 9, 0),
    "block": ("_ZN2gg3fp45block6kernel", 6, {4: 173}, 8, 8, 0),
    "tile": ("_ZN2gg3fp44tile6kernel", 4, {32: 276, 64: 304}, 21, 9, 72),
}


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    dst = tmp_path_factory.mktemp("isa") / "ragged_m_fp4.s"
    flags = [f for f in B.FLAGS if f != "-fPIC"]
    r = subprocess.run([B.HIPCC, *flags, "--cuda-device-only", "-S", f"{B.CSRC}/ragged_m_fp4.hip", "-o", str(dst)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    return dst.read_text()


@pytest.mark.parametrize("kernel", list(KERNELS))
def test_main_loop_budget(asm, kernel):
    prefix, instances, budget, loads, count, scratch = KERNELS[kernel]
    names = re.findall(r"^(" + prefix + r"\w+):", asm, re.M)
    assert len(names) == instances, names
    for name in names:
        seen = set()
        for label, ins in innermost_loops(asm, name):
            mfma = sum(x.startswith("v_mfma") for x in ins)
            if not mfma:
                continue
            seen.add(mfma)
            where = f"{name} {label}"
            assert mfma in budget and len(ins) <= budget[mfma], f"{where}: {len(ins)} instructions for {mfma} matrix instructions"
            memory = [x for x in ins if re.match(r"(scratch|global|flat|buffer)_", x)]
            assert all("offen lds" in x for x in memory), f"{where}: {[x for x in memory if 'offen lds' not in x]}"
            assert len(memory) == loads, f"{where}: {len(memory)} loads"
            waits = [int(n) for x in ins for n in re.findall(r"vmcnt\((\d+)\)", x)]
            assert waits == [count], f"{where}: waits for {waits}"
        assert seen == set(budget), f"{name}: loops of {seen} matrix instructions"
        size = re.search(r"; ScratchSize: (\d+)", asm[asm.index(".Lfunc_end", asm.index(f"\n{name}:")):])
        assert size and int(size.group(1)) <= scratch, f"{name}: {size and size.group(1)} scratch bytes per lane"
