"""What queries of the grouped products' status word return, in order, compiled for the host from the kernels' header."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, TIMEOUT = 0, 1, 6


def test_one_report_a_query_and_none_is_lost(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    exe = str(tmp_path / "status_harness")
    subprocess.run([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_103a,code=sm_103a",
                    "-I" + os.path.join(ROOT, "include"),
                    "-I" + os.path.join(ROOT, "nvfp4_quantization_grouped_gb300", "csrc"),
                    "-o", exe, os.path.join(ROOT, "tests", "native", "status_harness.cu")], check=True)
    out = subprocess.run([exe, "0", "1", "2", "3"], capture_output=True, text=True, check=True).stdout.split("\n")
    got = [[int(v) for v in line.split()] for line in out[:4]]
    assert got == [[OK], [INVALID, OK], [TIMEOUT, OK], [TIMEOUT, INVALID, OK]]
