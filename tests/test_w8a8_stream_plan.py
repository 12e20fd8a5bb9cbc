"""The sizes of the GPU tests of qlinear_w8a8's stream take it, with three tiles or more for a workgroup."""
from tests._w8_stream import STREAMS
from tests.test_w8a8_plan import _run, exe  # noqa: F401


def test_three_tiles_and_more(exe):  # noqa: F811
    slots = set()
    for M, N, K, _, shape in STREAMS:
        split, got, cuts, streamed = map(int, _run(exe, M, N, K, 0))
        assert (split, got, cuts) == (0, shape, 1) and streamed > 2 * 256, (M, N, K)
        slots.add((-(-K // 64) + 1) // 2 * 2 % 4)
    assert slots == {0, 2}
