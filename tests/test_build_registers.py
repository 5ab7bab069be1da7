"""What the built library's kernels take of the chip, by the notes that the
compiler leaves in their code: none keeps registers in memory."""
import os
import re
import shutil
import subprocess

import pytest

from moe_token_re_amd import _lib, build

LLVM = os.path.join(build.ROCM, "llvm", "bin")
TOOLS = [os.path.join(LLVM, t) for t in ("llvm-objdump", "llvm-readelf")]

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH) or not all(map(os.path.exists, TOOLS)),
                                reason="library not built, or no LLVM tools")


def kernels(tmp_path):
    """{kernel: {note: number}} of all code objects of the library."""
    lib = shutil.copy(_lib.LIB_PATH, tmp_path)
    subprocess.run([TOOLS[0], "--offloading", lib], cwd=tmp_path, check=True, stdout=subprocess.DEVNULL)
    found = {}
    for f in sorted(tmp_path.glob(f"*{build.ARCH}")):
        notes = subprocess.run([TOOLS[1], "--notes", f], check=True, capture_output=True, text=True).stdout
        for entry in re.split(r"^  - ", notes, flags=re.M)[1:]:
            name = re.search(r"^    \.symbol: +(\S+)\.kd", entry, flags=re.M)
            if name:
                found[name[1]] = {k: int(v) for k, v in re.findall(r"^    \.(\w+): +(\d+)$", entry, flags=re.M)}
    return found


def test_no_kernel_keeps_registers_in_memory(tmp_path):
    found = kernels(tmp_path)
    assert sum("few_up_kernel" in k for k in found) >= 7 and sum("grouped_mm_kernel" in k for k in found) == 6
    spilled = {k: v for k, v in found.items() if v["vgpr_spill_count"] or v["private_segment_fixed_size"]}
    assert not spilled, spilled
