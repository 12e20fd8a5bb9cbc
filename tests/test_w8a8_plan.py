"""Which kernel takes a qlinear_w8a8 call (csrc/w8a8_plan.h, the source that the
launch compiles) built for the host: over many sizes what it plans exists and
covers the outputs, and the GPU tests' sizes take every way there is."""
import os
import shutil
import subprocess

import pytest

import mixed_precision_quantized_act_amd as qa
from tests._w8 import PLANS

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mixed_precision_quantized_act_amd", "csrc")


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    out = tmp_path_factory.mktemp("w8a8") / "w8a8_plan_check"
    subprocess.run([cxx, "-O2", "-std=c++17", "-Wall", "-Werror", "-I", CSRC,
                    os.path.join(ROOT, "tests", "w8a8_plan_check.cpp"), "-o", str(out)],
                   check=True, capture_output=True, text=True)
    return str(out)


def _run(exe, *args):
    r = subprocess.run([exe, *map(str, args)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout
    return r.stdout.split()


def test_many_sizes(exe):
    assert _run(exe)[0] == "ok"


@pytest.mark.parametrize("kind", list(PLANS))
def test_the_sizes_of_the_gpu_tests(exe, kind):
    for M, N, K in PLANS[kind]:
        ws = qa.qlinear_w8a8_workspace(M, N, K)
        split, shape, cuts, streamed = map(int, _run(exe, M, N, K, ws))
        assert (split, shape, int(cuts > 1), int(streamed > 0)) == kind, (M, N, K)
        assert (ws > 0) == (cuts > 1)


def test_without_a_workspace_nothing_is_cut(exe):
    for sizes in PLANS.values():
        for M, N, K in sizes:
            assert _run(exe, M, N, K, 0)[2] == "1"
