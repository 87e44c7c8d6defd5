"""Host checks of the kernels' own rules for the cache, attention and sampling (no GPU)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_numbers_in_device_memory(tmp_path):
    # Row starts whose difference wraps around among them: no row outside the matrices is taken for a sequence's own.
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    exe = str(tmp_path / "seq_rows_test")
    subprocess.check_call([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_103a,code=sm_103a",
                           os.path.join(ROOT, "tests", "seq_rows_host_test.cu"), "-o", exe])
    run = subprocess.run([exe], capture_output=True, text=True)
    assert run.returncode == 0 and "PASS" in run.stdout, run.stdout
