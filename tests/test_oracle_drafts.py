"""The oracle of a checked step of drafted tokens against worked examples."""
import numpy as np
import pytest

from oracle import drafts as O


def test_sums_of_codes():
    a, w = np.array([[-128, 127, 3]], np.int8), np.array([[-128, -128, 1], [127, 127, 0]], np.int8)
    assert O.int8_sums(a, w).tolist() == [[16384 - 16256 + 3, -16256 + 16129]]


def test_a_quarter_turn():
    x = np.arange(1.0, 9.0).reshape(1, 1, 8)
    f = np.array([np.pi / 2, 0.0])
    assert np.allclose(O.turn(x, 4, 1, f, 1.0, [1]), [[[-2, 1, 3, 4, 5, 6, 7, 8]]])
    assert np.allclose(O.turn(x, 4, 2, f, 2.0, [1]), [[[-6, 4, 2, 8, 5, 6, 7, 8]]])
    assert np.array_equal(O.turn(x, 4, 2, f, 2.0, [-1]), x)


def test_frequencies():
    assert np.allclose(O.frequencies(4, 10000.0, 0, 1.0)[0], [1.0, 0.01])
    assert np.allclose(O.frequencies(4, 10000.0, 1, 4.0)[0], [0.25, 0.0025])
    f, s = O.frequencies(64, 10000.0, 2, 8.0)                  # the last pair exactly 8 times slower
    assert f[0] == 1.0 and np.isclose(f[-1], 10000.0 ** (-62 / 64) / 8.0) and s == 1.0
    f, s = O.frequencies(128, 10000.0, 3, 16.0, 4096.0)
    plain = O.frequencies(128, 10000.0, 0, 1.0)[0]
    turns = 4096 * plain / (2 * np.pi)
    assert np.allclose(f[turns > 40], plain[turns > 40]) and np.allclose(f[turns < 0.8], plain[turns < 0.8] / 16)
    assert np.isclose(s, 0.1 * np.log(16.0) + 1)
    assert np.all(np.diff(f) < 0)


def test_a_tree():
    #   0 -> 1 -> 3, 0 -> 2; 4 alone
    seen = O.ancestors([-1, 0, 0, 1, -1])
    assert [np.flatnonzero(r).tolist() for r in seen] == [[0], [0, 1], [0, 2], [0, 1, 3], [4]]
    assert O.words(seen).ravel().tolist() == [1, 3, 5, 11, 16]
    assert np.flatnonzero(O.tree_sees(seen, 5, 7)[3]).tolist() == [0, 1, 2, 3, 5]
    assert np.flatnonzero(O.tree_sees(seen, 5, 3)[3]).tolist() == [1]         # nodes 0 and 1 have no position


@pytest.mark.parametrize("T", [1, 63, 64, 65, 130])
def test_words_bit_by_bit(T):
    seen = np.random.default_rng(T).random((T, T)) < 0.4
    w = O.words(seen).view(np.uint64)
    assert w.shape == (T, -(-T // 64))
    for i in range(T):
        for j in range(w.shape[1] * 64):
            assert bool((int(w[i, j // 64]) >> (j % 64)) & 1) == (j < T and bool(seen[i, j]))


def test_keep_reads_before_it_writes():
    class C:
        k_q = np.arange(8, dtype=np.uint8).reshape(2, 1, 4, 1)
        k_s, v_q, v_s = k_q + 10, k_q + 20, k_q + 30

        @staticmethod
        def slot(b, pos):
            return (pos // 4, pos % 4) if 0 <= pos < 7 else None
    O.keep(C, [1], [[1, 0, 0, 5, 9]], [5])       # a swap, the same token twice, one moved back, one without a slot
    assert C.k_q.ravel().tolist() == [0, 2, 1, 1, 6, 5, 6, 7]
    assert C.v_s.ravel().tolist() == [30, 32, 31, 31, 36, 35, 36, 37]
