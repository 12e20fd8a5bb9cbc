"""How attention of few rows is laid out (csrc/attn_few_plan.h, the source that the launch compiles) built for the host:
over many sizes, and the workspace that a tree's call asks for is that of its own plan."""
import os
import shutil
import subprocess

import pytest

import mixed_precision_quantized_act_amd as qa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mixed_precision_quantized_act_amd", "csrc")


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    out = tmp_path_factory.mktemp("few") / "attn_few_plan_check"
    subprocess.run([cxx, "-O2", "-std=c++17", "-Wall", "-Werror", "-I", CSRC,
                    os.path.join(ROOT, "tests", "attn_few_plan_check.cpp"), "-o", str(out)],
                   check=True, capture_output=True, text=True)
    return str(out)


def _run(exe, *args):
    r = subprocess.run([exe, *map(str, args)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
    return r.stdout.split()


def test_many_sizes(exe):
    assert _run(exe)[0] == "ok"


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,T,Hq,H,L", [(16, 8, 32, 8, 32768), (16, 16, 32, 8, 32768), (1, 17, 128, 128, 16000), (5, 13, 24, 8, 4099),
                                        (16, 1, 32, 8, 32768), (16, 10, 32, 8, 32768), (64, 8, 32, 8, 4096), (4, 64, 16, 16, 32768)])
def test_a_tree_asks_for_what_its_plan_takes(exe, B, T, Hq, H, L, D):
    sets, tiles, splits = map(int, _run(exe, 1, B, T, Hq, H, D, L))
    asked = qa.attn_kv4_tree_workspace(B, T, Hq, H, D, L)
    assert asked == (splits * B * T * Hq * (D + 2) * 4 if splits > 1 else 0)
    # the other calls: one sixteen a wave
    sets, tiles, splits = map(int, _run(exe, 0, B, T, Hq, H, D, L))
    assert sets == 1
    if T * (Hq // H) < 64:
        assert qa.attn_kv4_workspace(B, T, Hq, H, D, L) == (splits * B * T * Hq * (D + 2) * 4 if splits > 1 else 0)
