"""The gradient-list and cross-entropy calls from plain C: the header stays
strict C99 and the library exports what it declares."""
import os
import shutil
import subprocess

import pytest

import loss_scaled_fp32_b200 as lsf

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_plain_c_consumer_of_the_operators(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no gcc")
    lib_dir = os.path.dirname(lsf.lib()._name)
    exe = str(tmp_path / "abi_operators")
    build = subprocess.run(
        [gcc, "-std=c99", "-Wall", "-Wextra", "-Wpedantic", "-Werror", "-I", os.path.join(ROOT, "include"),
         os.path.join(ROOT, "tests", "native", "abi_operators.c"), "-L", lib_dir, "-lmpt",
         "-Wl,-rpath," + lib_dir, "-o", exe], capture_output=True, text=True)
    assert build.returncode == 0, build.stderr
    run = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, run.stderr
    assert "10 entry points" in run.stdout
