"""How the operators around the scan choose their kernels (csrc/ssd_step.hpp),
driven by tests/native/step_choice_check.cpp (CPU only)."""
import os
import shutil

import pytest


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_choice_of_kernels(tmp_path):
    # (imported here: the file may be left out where only the GPU tests run)
    from test_native_sanitizers import CSRC, NATIVE, ROOT, _build_and_run
    out = _build_and_run(
        tmp_path, "g++", [os.path.join(NATIVE, "step_choice_check.cpp")],
        ["-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
         "-I", os.path.join(ROOT, "include"), "-I", CSRC], "step_choice_check")
    assert "0 failed expectations" in out
