"""Attention of many rows whose keys are cut unevenly among the workgroups
(tests/test_attn_cuts.py says that these sizes are), against float64."""
import pytest

from tests._cuts import CASES
from tests.test_gpu_attn import _cross, _kv4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("name", [n for n in CASES if CASES[n]["L"] <= 2000])
def test_cache(name, causal):
    c = CASES[name]
    # a stream that ends within the table's last tile, and one well before it
    lens = [c["L"] - 10, 700][:c["B"]]
    _kv4(41, c["B"], c["Lq"], c["Hq"], c["H"], c["D"], 64, lens, causal=causal, extra_pages=0)


@pytest.mark.parametrize("name", list(CASES))
def test_states(name):
    c = CASES[name]
    k_lens = [c["L"] - 5, 1000][:c["B"]]
    _cross(41, c["B"], c["Lq"], c["L"], c["Hq"], c["H"], c["D"], k_lens=k_lens)


def test_states_that_end_with_the_last_piece():
    """Every state seen, and the last state alone."""
    c = CASES["86 heads of 64, 1600 keys"]
    _cross(42, 1, c["Lq"], c["L"], c["Hq"], c["H"], c["D"])
    import numpy as np
    m = np.zeros((1, c["L"]), bool)
    m[0, -1] = True
    _cross(42, 1, c["Lq"], c["L"], c["Hq"], c["H"], c["D"], mask=m)
