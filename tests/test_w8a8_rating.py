"""What qlinear_w8a8's plan rates itself at (csrc/w8a8_plan.h built for the host) against times and rates of an MI355X."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mixed_precision_quantized_act_amd", "csrc")
MOST = 1.06 * 2.50e15      # operations a second: the longest K reaches 2.50e15, 8192^3 2.43e15
# us, one call among others, bf16 outputs
TIMES = [(8192, 8192, 16384, 880), (8192, 8192, 8192, 452), (8192, 8192, 4096, 243), (8192, 8192, 2048, 138),
         (16384, 8192, 4096, 475), (17776, 5760, 1920, 203), (17776, 1920, 7680, 247), (17776, 7680, 1920, 259),
         (4096, 4096, 8192, 116), (4096, 4096, 4096, 63.3), (4096, 4096, 2048, 35.5), (4096, 4096, 1024, 21.4)]


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    out = tmp_path_factory.mktemp("w8a8") / "w8a8_rating_check"
    subprocess.run([cxx, "-O2", "-std=c++17", "-Wall", "-Werror", "-I", CSRC,
                    os.path.join(ROOT, "tests", "w8a8_rating_check.cpp"), "-o", str(out)],
                   check=True, capture_output=True, text=True)
    return str(out)


@pytest.mark.parametrize("M,N,K,us", TIMES)
def test_rated_as_measured(exe, M, N, K, us):
    rated = float(subprocess.run([exe, str(M), str(N), str(K)], capture_output=True, text=True, check=True).stdout)
    assert 2.0 * M * N * K / (rated * 1e-6) <= MOST
    assert abs(rated / us - 1) <= 0.15
