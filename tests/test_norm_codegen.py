"""The workgroups of a CU that the plan of the layer norm's backward pass counts on, against the registers of the compiled
kernels."""
import os
import re
import shutil
import subprocess

import pytest

from selective_state_space_75_amd import build as B

pytestmark = pytest.mark.skipif(not (os.path.exists(B.HIPCC) or shutil.which(B.HIPCC)), reason="no HIP compiler")

REGISTERS = 512                        # of a SIMD's lane, in eights a wave; four SIMDs a CU
TYPES = {"kNormBwd2": ("tt",), "kNormBwd4": ("tf", "ft", "ff")}        # x's and dy's: t 2 bytes, f 4


def tables():
    with open(os.path.join(B.PKG, "csrc", "kernels.hpp"), encoding="utf-8") as f:
        text = f.read()
    return {n: [tuple(map(int, re.findall(r"\d+", s))) for s in re.findall(r"\{(\d+(?:, \d+){4})\}", row)]
            for n, row in re.findall(r"(kNormBwd\d)\[\w+\] = \{(.*)\};", text)}


def test_the_plan_counts_on_what_the_registers_hold(tmp_path):
    out = str(tmp_path / "layer_norm_bwd.s")
    subprocess.run([B.HIPCC] + B.FLAGS + ["-I", os.path.join(B.ROOT, "include"), "-I", os.path.join(B.PKG, "csrc"),
                                          "--cuda-device-only", "-S", "-o", out, os.path.join(B.PKG, "csrc", "layer_norm_bwd.hip")],
                   check=True, capture_output=True)
    with open(out, encoding="utf-8") as f:
        text = f.read()
    used, spilled = {}, []
    for block in text.split("amdhsa.kernels:")[1].split("  - .agpr_count:")[1:]:
        agprs, name = int(block.split()[0]), re.search(r"\.name:\s+(\S+)", block).group(1)
        count = agprs + int(re.search(r"\.vgpr_count:\s+(\d+)", block).group(1))
        if int(re.search(r"\.vgpr_spill_count:\s+(\d+)", block).group(1)):
            spilled.append(name)
        m = re.search(r"norm_col_bwd_kernelI(\w\w)Lb([01])ELi(\d+)ELi(\d+)ELi(\d+)E", name)
        if m:
            used[m.group(1), int(m.group(2))] = {**used.get((m.group(1), int(m.group(2))), {}),
                                                 tuple(map(int, m.groups()[2:])): count}
    assert not spilled, spilled
    off = {}
    for table, shapes in tables().items():
        assert len(shapes) == 3
        for threads, lanes, chans, *planned in shapes:
            for gate in (0, 1):
                held = min(REGISTERS // (-(-used[t, gate][threads, lanes, chans] // 8) * 8) * 256 // threads for t in TYPES[table])
                if held != planned[gate]:
                    off[table, threads, lanes, chans, gate] = (held, planned[gate])
    # counted on one more, as measured (beside the table)
    assert off == {("kNormBwd4", 256, 4, 2, 1): (3, 4)}
