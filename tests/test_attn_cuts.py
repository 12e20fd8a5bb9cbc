"""The cut of the keys among workgroups (csrc/attn_cuts.h, the source that the
attention tiles' launch compiles) built for the host."""
import os
import shutil
import subprocess

import pytest

from tests._cuts import CASES, row_tiles

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mixed_precision_quantized_act_amd", "csrc")


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    out = tmp_path_factory.mktemp("cuts") / "attn_cuts_check"
    subprocess.run([cxx, "-O2", "-std=c++17", "-Wall", "-Werror", "-I", CSRC,
                    os.path.join(ROOT, "tests", "attn_cuts_check.cpp"), "-o", str(out)],
                   check=True, capture_output=True, text=True)
    return str(out)


def _plan(exe, u, rows, D, tiles, fit):
    r = subprocess.run([exe] + [str(x) for x in (u, rows, D, tiles, fit)], check=True, capture_output=True, text=True)
    return tuple(int(x) for x in r.stdout.split())


def test_every_cut_is_what_its_plan_says(exe):
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:]
    assert " 0 failures" in r.stdout


def test_twenty_row_tiles(exe):
    """Twelve equal pieces (240 workgroups at once); thirteen pieces with a
    smaller last one would leave 16 places for its 20."""
    assert _plan(exe, 20, 4 * 1137, 64, 259, 1000) == (12, 1, 12)


@pytest.mark.parametrize("name", list(CASES))
def test_the_uneven_cases_are_uneven(exe, name):
    """What the GPU's test of uneven pieces takes for granted."""
    c = CASES[name]
    n, size, whole = _plan(exe, row_tiles(c), c["B"] * c["Lq"] * c["Hq"], c["D"], -(-c["L"] // 64), 1000)
    assert n > 1 and size * n != whole and (n, size) == c["cut"]
