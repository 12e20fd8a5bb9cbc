"""kv4_keep against the oracle's moves, byte by byte."""
import numpy as np
import pytest

from oracle import drafts as O
from tests._attn import CacheCase, rng
from tests._gpu import dev, host, torch

pytestmark = pytest.mark.gpu


def _qa():
    import mixed_precision_quantized_act_amd as qa
    return qa


def _keep(seed, B, T, H, D, page, start, path, count=None, **kw):
    qa, t = _qa(), torch()
    case = CacheCase(seed, B, H, D, page, kw.pop("lens", [max(1, s + T) for s in start]), **kw)
    path = np.asarray(path, np.int32).reshape(B, T)
    k_q, k_s, v_q, v_s, _, _, table = case.device(dev)
    qa.kv4_keep(k_q, k_s, v_q, v_s, table, dev(np.asarray(start, np.int32)), dev(path), B, T,
                count=None if count is None else dev(np.asarray(count, np.int32)))
    t.cuda.synchronize()
    c = case.cache
    O.keep(c, start, path.astype(np.int64), [T] * B if count is None else [min(max(n, 0), T) for n in count])
    for got, want in zip((k_q, k_s, v_q, v_s), (c.k_q, c.k_s, c.v_q, c.v_s)):
        np.testing.assert_array_equal(host(got), want)


def _paths(seed, B, T):
    """Rising ones, as a checked tree leaves them."""
    g = rng(721, seed, B, T)
    return np.stack([np.sort(g.choice(T, T, replace=True)) for _ in range(B)])


@pytest.mark.parametrize("D", [16, 48, 64, 80, 128, 256])
@pytest.mark.parametrize("page", [16, 64])
def test_heads_and_pages(D, page):
    _keep(1, 3, 11, 3, D, page, [0, page - 2, 3 * page + 1], _paths(1, 3, 11))


@pytest.mark.parametrize("B,T,H", [(1, 1, 1), (37, 1, 8), (1, 250, 6), (4, 33, 5), (2, 256, 1), (1, 257, 2), (1, 700, 1),
                                   (1, 1024, 2)])
@pytest.mark.parametrize("D", [64, 256])
def test_sizes(B, T, H, D):
    _keep(2, B, T, H, D, 32, [(7 * b) % 90 for b in range(B)], _paths(2, B, T))


@pytest.mark.parametrize("T", [2, 40, 300, 1024])
def test_any_order_and_the_same_place_twice(T):
    g = rng(722, T)
    _keep(3, 2, T, 2, 64, 16, [5, 30], np.stack([g.permutation(T), np.arange(T)[::-1]]))
    _keep(3, 2, T, 2, 64, 16, [5, 30], g.integers(0, T, (2, T)))
    _keep(3, 2, T, 2, 128, 64, [0, 64], np.stack([np.roll(np.arange(T), 1), np.zeros(T, int)]))


def test_counts_and_places_without_a_slot():
    path = rng(723).integers(0, 20, (6, 20))
    path[3, 4], path[3, 5], path[4, 2] = 10 ** 6, -2 ** 31, -7           # past the table, no position, before the start
    _keep(4, 6, 20, 2, 64, 16, [5, 10, 20, 45, 9, -3], path, count=[0, 20, 7, 20, 20, 20], lens=[25, 30, 40, 65, 29, 17],
          bad=((1, 1, -1), (2, 2, 10 ** 6)))
    _keep(4, 3, 20, 2, 64, 16, [5, 10, 2 ** 31 - 1], path[:3], count=[-1, 100, 20], lens=[25, 30, 40])


def test_no_tokens_and_gate():
    qa, t = _qa(), torch()
    case = CacheCase(6, 2, 2, 64, 16, [25, 29])
    k_q, k_s, v_q, v_s, _, _, table = case.device(dev)
    st, path = dev(np.array([5, 9], np.int32)), dev(np.arange(40, dtype=np.int32)[::-1].copy() % 20).view(2, 20)
    qa.kv4_keep(k_q, k_s, v_q, v_s, table, st, path[:, :0].contiguous(), 2, 0)
    with qa.gate(t.zeros(1, dtype=t.uint8, device="cuda"), 1):
        qa.kv4_keep(k_q, k_s, v_q, v_s, table, st, path, 2, 20)
    t.cuda.synchronize()
    for p, q in zip((k_q, k_s, v_q, v_s), (case.cache.k_q, case.cache.k_s, case.cache.v_q, case.cache.v_s)):
        assert np.array_equal(host(p), q)


def test_captured_and_replayed():
    qa, t = _qa(), torch()
    case = CacheCase(7, 2, 2, 64, 16, [80, 90])
    parts = case.device(dev)
    st, count = dev(np.array([60, 70], np.int32)), dev(np.array([5, 9], np.int32))
    path = dev(_paths(7, 2, 20).astype(np.int32))
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        qa.kv4_keep(*parts[:4], parts[6], st, path, 2, 20, count=count)
    for i in range(4):
        p = _paths(8 + i, 2, 20)
        path.copy_(dev(p.astype(np.int32)))
        count.copy_(dev(np.array([i, 20 - i], np.int32)))
        graph.replay()
        t.cuda.synchronize()
        O.keep(case.cache, [60, 70], p, [i, 20 - i])
        c = case.cache
        for got, want in zip(parts, (c.k_q, c.k_s, c.v_q, c.v_s)):
            np.testing.assert_array_equal(host(got), want)
