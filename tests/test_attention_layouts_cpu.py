"""What attention's argument checks say of tensors that interleave, against a
count of every element they hold (a C++ program, on the CPU).
"""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_shared_memory_is_found_and_slices_are_told_apart(tmp_path):
    exe = os.path.join(tmp_path, "layouts_check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror",
                    "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "diffusion_transformer_qk_amd", "csrc"),
                    os.path.join(ROOT, "tests", "c_abi", "layouts_check.cpp"), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout + out.stderr
