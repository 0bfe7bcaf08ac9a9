"""The layer operators' host layer (``layer_api.cpp``) under AddressSanitizer
and UndefinedBehaviorSanitizer (CPU only): built with g++ against launchers
that abort if reached and driven over random shapes and row strides with
extreme values."""
import os
import shutil

import pytest

from test_host_sanitizers import CSRC, ENV, HERE, ROOT, SAN, _run

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="host compiler not available")


def test_layer_abi_host_layer_under_asan_ubsan(tmp_path):
    exe = str(tmp_path / "layer_driver")
    _run(["g++", "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
          "-I", "/opt/rocm/include", os.path.join(CSRC, "layer_api.cpp"), os.path.join(HERE, "sanitize", "layer_stubs.cpp"),
          os.path.join(HERE, "sanitize", "layer_driver.cpp"), "-L", "/opt/rocm/lib", "-lamdhip64",
          "-Wl,-rpath,/opt/rocm/lib", "-o", exe])
    r = _run([exe, "60000"], env=ENV, timeout=600)
    print(r.stdout)
    assert ", 0 mismatches" in r.stdout and ", 0 valid" not in r.stdout
