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


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_tile_shapes_of_products(tmp_path):
    """The sizes of the GPU test of every tile do reach every tile, in both
    types; a refit that loses one has to bring sizes for it."""
    import subprocess

    from test_gpu_linear import TILES
    from test_gpu_linear_plans import TWICE
    from test_native_sanitizers import CSRC, NATIVE, ROOT, _build_and_run
    _build_and_run(
        tmp_path, "g++", [os.path.join(NATIVE, "linear_choice_check.cpp")],
        ["-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
         "-I", os.path.join(ROOT, "include"), "-I", CSRC], "linear_choice_check")
    for bf16, shapes in ((1, 13), (0, 10)):
        sizes = "".join(f"{bf16} {M} {N} {K}\n" for M, N, K in TILES)
        out = subprocess.run([str(tmp_path / "linear_choice_check")], input=sizes,
                             capture_output=True, text=True, timeout=60, check=True).stdout
        plans = [tuple(map(int, line.split()[1:])) for line in out.splitlines()
                 if line.startswith("plan")]
        assert len(plans) == len(TILES)
        missing = set(range(shapes)) - {s for p in plans for s in p}
        assert not missing, (bf16, missing)
        assert len({a for a, b in plans if b < 0}) >= 5
        sizes = "".join(f"{bf16} {M} {N} {K}\n" for M, N, K in TWICE[bf16])
        out = subprocess.run([str(tmp_path / "linear_choice_check")], input=sizes,
                             capture_output=True, text=True, timeout=60, check=True).stdout
        twice = [line.split()[1:] for line in out.splitlines() if line.startswith("plan")]
        assert len(twice) == len(TWICE[bf16]) and all(b != "-1" for _, b in twice), twice
