"""The recurrence's kernels hold their tiles in registers without spilling any: vector
registers saved to memory at a place where some lanes are switched off come back wrong (seen
with this compiler, in a kernel that stored a block's scale from some of its lanes).  Read
from the metadata of the objects that the build leaves."""
import os
import re
import subprocess

import pytest

from selective_state_space_sscan_amd import build as B

LLVM = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin")


@pytest.mark.parametrize("source", [s for s in B.SOURCES if s.startswith(("sscan_rec", "sscan_pack8", "sscan_layer"))
                                    and s.endswith(".hip")])
def test_no_vector_register_is_spilled(source, tmp_path):
    bundler, readelf = (os.path.join(LLVM, n) for n in ("clang-offload-bundler", "llvm-readelf"))
    if not (os.path.exists(bundler) and os.path.exists(readelf)):
        pytest.skip("LLVM's tools are not installed")
    obj = os.path.join(B.OBJ_DIR, os.path.splitext(source)[0] + ".o")
    if not os.path.exists(obj):
        B.build(force=False)
    fat, code = str(tmp_path / "fat.bin"), str(tmp_path / "code.o")
    subprocess.run([os.path.join(LLVM, "llvm-objcopy"), f"--dump-section=.hip_fatbin={fat}", obj, os.devnull], check=True)
    subprocess.run([bundler, "--unbundle", "--type=o", "--targets=hipv4-amdgcn-amd-amdhsa--gfx950", f"--input={fat}",
                    f"--output={code}"], check=True)
    notes = subprocess.run([readelf, "--notes", code], check=True, capture_output=True, text=True).stdout
    kernels = re.findall(r"\.name:\s+(_Z\S+)$.*?\.vgpr_spill_count:\s+(\d+)", notes, re.M | re.S)
    assert kernels
    assert [k for k, n in kernels if int(n)] == []
