"""The gated delta rule's and the norms' argument checks under AddressSanitizer and
UndefinedBehaviorSanitizer (host code only, CPU): sscan_delta_capi.cpp is compiled with
them, linked with the library's other objects and driven by test_delta_abi_cpu.py."""
import glob
import os
import subprocess

import pytest

from selective_state_space_sscan_amd import build as B
from test_asan_host import _run_tests


def test_delta_abi_checks_under_asan_ubsan(tmp_path):
    rts = glob.glob("/opt/rocm/llvm/lib/clang/*/lib/linux/libclang_rt.asan-x86_64.so")
    if not rts:
        pytest.skip("clang's AddressSanitizer runtime is not installed")
    objs = [os.path.join(B.OBJ_DIR, os.path.splitext(s)[0] + ".o") for s in B.SOURCES if s != "sscan_delta_capi.cpp"]
    if not all(os.path.exists(o) for o in objs):
        B.build(force=False)
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined"]
    capi, lib = str(tmp_path / "sscan_delta_capi.o"), str(tmp_path / "libsscan_asan.so")
    common = ["--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-fno-omit-frame-pointer",
              "-fvisibility=hidden", "-I", B.INCLUDE, "-I", B.CSRC]
    subprocess.run([B.hipcc()] + common + san + ["-c", "-o", capi, os.path.join(B.CSRC, "sscan_delta_capi.cpp")],
                   check=True, capture_output=True)
    subprocess.run([B.hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC"] + san + ["-o", lib, capi] + objs,
                   check=True, capture_output=True)
    _run_tests(["tests/test_delta_abi_cpu.py"], {"SSCAN_TEST_LIBRARY": lib, "LD_PRELOAD": rts[0]}, tmp_path)
