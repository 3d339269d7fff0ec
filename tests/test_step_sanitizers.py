"""The C ABI layer of the operators around the scan (csrc/ssd_step_api.cpp)
under AddressSanitizer and UndefinedBehaviorSanitizer, driven by
tests/native/step_host_check.cpp against stand-ins for the launchers (CPU
only; no device code is built here)."""
import os
import shutil

import pytest


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_step_layer_under_sanitizers(tmp_path):
    # (imported here: the file may be left out where only the GPU tests run)
    from test_native_sanitizers import CSRC, NATIVE, ROOT, _build_and_run
    out = _build_and_run(
        tmp_path, "g++",
        [os.path.join(CSRC, "ssd_step_api.cpp"), os.path.join(NATIVE, "step_host_check.cpp")],
        ["-std=c++17", "-DSSD_DEBUG_CHECKS", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
         "-I", os.path.join(ROOT, "include"), "-I", CSRC], "step_host_check")
    assert "0 failed expectations" in out
