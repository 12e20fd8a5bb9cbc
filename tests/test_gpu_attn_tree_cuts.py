"""attn_kv4_tree's kernels of many rows: whole units, equal pieces of their keys and shares of the list of all
streams' tiles.  The work is laid out for the table's length, so a long table with short streams reaches them."""
import numpy as np
import pytest

from oracle import drafts as O
from tests._attn import CacheCase, rng
from tests._gpu import dev, torch
from tests.test_gpu_attn_tree import _qa, _tree, _trees, _ws

pytestmark = pytest.mark.gpu


def _kind(B, T, Hq, H, D, cols):
    """Which cut the workspace's size tells of (shares' sums and units'; n pieces of a unit, one each)."""
    rows = T * (Hq // H)
    assert rows > 48 and B * H * -(-rows // 16) * -(-cols // 64) > 6 * 1024
    assert rows > 64 or B * H * -(-rows // 16) * -(-cols // 64) < 64 * 1024
    tile = 128 if rows <= 128 else 256
    units, n = B * H * -(-rows // tile), _qa().attn_kv4_tree_workspace(B, T, Hq, H, D, cols)
    if n == 0:
        return "whole"
    if n % (units * tile * (D + 2) * 4) == 0:
        return "pieces"
    shares = (n - units * 8) // (tile * (D + 2) * 4) - units
    assert 128 <= shares <= 256 and (n - units * 8) % (tile * (D + 2) * 4) == 0
    return "shares"


def _cols(lens, extra, page):
    return (max(-(-max(1, n) // page) for n in lens) + extra) * page


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,kind", [(49, "tree"), (64, "bits"), (65, "tree"), (128, "bits"), (129, "tree"), (257, "bits")])
def test_shares(D, T, kind):
    lens = [1500, T, T + 70]
    assert _kind(3, T, 1, 1, D, _cols(lens, 800, 64)) == "shares"
    _tree(21, 3, T, 1, 1, D, 64, lens, kind=kind, extra_pages=800)


@pytest.mark.parametrize("T,D", [(60, 128), (200, 64)])
def test_any_workspace(T, D):
    for ws in (0, 100_000, 5_000_000):
        _tree(22, 2, T, 1, 1, D, 64, [1000, T], extra_pages=1000, ws=ws, pad=8)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,Hq,H", [(66, 3, 3), (33, 6, 2), (140, 1, 1)])
def test_streams_of_all_lengths(D, T, Hq, H):
    """Without positions, without tokens, with fewer positions than tokens, of one tile, of many."""
    lens = [0, 500, 20, 64, 2500, 1, T, 1100, 300, 65]
    q_lens = [T, 0, T, T, T, 1, T, T - 1, 17, 2]
    assert _kind(10, T, Hq, H, D, _cols(lens, 1000, 32)) == "shares"
    _tree(23, 10, T, Hq, H, D, 32, lens, q_lens=q_lens, extra_pages=1000)
    _tree(23, 10, T, Hq, H, D, 32, lens, q_lens=q_lens, kind="bits", shared=True, extra_pages=1000)


def test_no_stream_has_tokens():
    T = 70
    _tree(24, 3, T, 1, 1, 64, 64, [100, 0, 500], q_lens=[0, 0, 0], extra_pages=800)


def test_shares_of_many_tiles():
    """Begins of shares that move to a unit's."""
    lens = [8192, 8000, 333, 6000]
    assert _kind(4, 66, 4, 4, 128, _cols(lens, 512, 64)) == "shares"
    _tree(25, 4, 66, 4, 4, 128, 64, lens, extra_pages=512)


def test_more_streams_than_lanes():
    g = rng(713)
    for B in (65, 130):
        lens = [int(x) for x in g.integers(0, 200, B)]
        q_lens = [int(x) for x in g.integers(0, 66, B)]
        assert _kind(B, 65, 1, 1, 64, _cols(lens, 720, 32)) == "shares"
        _tree(26, B, 65, 1, 1, 64, 32, lens, q_lens=q_lens, extra_pages=720)


@pytest.mark.parametrize("T,D", [(65, 64), (130, 64), (70, 128)])
def test_whole_units(T, D):
    lens, q_lens = [T, 300, 1, 0, 40, 150, 64, 77], [T, T, 3, T, 0, T - 1, T, 20]
    assert _kind(8, T, 32, 32, D, _cols(lens, 10, 64)) == "whole"
    _tree(27, 8, T, 32, 32, D, 64, lens, q_lens=q_lens, extra_pages=10)


@pytest.mark.parametrize("T,D", [(100, 128), (60, 128)])
def test_equal_pieces(T, D):
    lens, q_lens = [T, 900, 1, 0, 40, 2000, 64, 77], [T, T, 3, T, 0, T - 1, T, 20]
    assert _kind(8, T, 8, 8, D, _cols(lens, 92, 64)) == "pieces"
    _tree(28, 8, T, 8, 8, D, 64, lens, q_lens=q_lens, extra_pages=92)
    _tree(28, 8, T, 8, 8, D, 64, lens, q_lens=q_lens, extra_pages=92, ws=9_000_000, kind="bits")


def test_pages_without_a_place():
    bad = ((0, 1, -1), (0, 2, 10 ** 8), (1, 0, -2 ** 31), (1, 6, -5), (1, 40, -1))
    for T, D in ((60, 64), (100, 128), (200, 64), (150, 128)):
        _tree(29, 2, T, 1, 1, D, 32, [2000, 1500], bad=bad, extra_pages=2500)
        _tree(29, 2, T, 1, 1, D, 32, [200, 210], bad=bad, kind="bits", extra_pages=2500)


@pytest.mark.parametrize("gain,scale", [(60.0, None), (1e-3, None), (1.0, 3.0), (1.0, 1e-6)])
def test_sizes_of_queries_and_scale(gain, scale):
    for T, D in ((60, 64), (150, 128)):
        _tree(30, 2, T, 1, 1, D, 32, [700, 300], gain=gain, scale=scale, extra_pages=2500)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,extra", [(3, 1), (20, 1), (60, 1500), (200, 1500)])
def test_a_token_that_a_row_does_not_see_may_hold_any_bytes(D, T, extra):
    """NaN's scales of one drafted token: the rows of the others as without."""
    qa, t = _qa(), torch()
    B, n = 2, T + 333
    case = CacheCase(31, B, 1, D, 64, [n, n], extra_pages=extra)
    q = t.randn((B * T, 2 * D), device="cuda", generator=t.Generator(device="cuda").manual_seed(6)).bfloat16()
    word, lens = dev(O.words(O.ancestors([-1] * T))), dev(np.array([n, n], np.int32))
    nws = qa.attn_kv4_tree_workspace(B, T, 2, 1, D, case.cache.table.shape[1] * 64)
    out = []
    for bad in (None, 0x7F, 0xFF):
        parts = case.device(dev)
        if bad is not None:
            p = n - T + T // 2
            page = int(case.cache.table[0, p // 64])
            parts[1][page, 0, p % 64] = bad
            parts[3][page, 0, p % 64] = bad
        o = t.empty_like(q)
        qa.attn_kv4_tree(q, *parts, lens, word, o, B, T, 2, ws=_ws(nws))
        out.append(o)
    mask = t.ones_like(q, dtype=t.bool)
    mask[T // 2] = False
    for o in out[1:]:
        assert t.equal(o[mask], out[0][mask])


@pytest.mark.parametrize("D,T", [(64, 60), (128, 100), (64, 200), (128, 150)])
def test_captured_and_replayed_beside_another(D, T):
    """Lengths that change between replays change the shares; another stream's call has its own workspace."""
    qa, t = _qa(), torch()
    g = rng(714, T)
    case = CacheCase(32, 2, 2, D, 64, [5000, 3000], extra_pages=500)
    parts = case.device(dev)
    n = qa.attn_kv4_tree_workspace(2, T, 2, 2, D, case.cache.table.shape[1] * 64)
    sets = [(t.randn((2 * T, 2 * D), device="cuda").bfloat16(), dev(np.array(ln, np.int32)), dev(np.array(m, np.int32)),
             dev(O.words(_trees(g, 2, T, "tree")))) for ln, m in (([5000, 3000], [T, T]), ([T, 200], [T, 1]), ([900, 2991], [3, T]))]
    want = []
    for q, ln, m, word in sets:
        o = t.zeros_like(q)
        qa.attn_kv4_tree(q, *parts, ln, word, o, 2, T, 2, q_lens=m, ws=_ws(n))
        want.append(o)
    held, o, ws = [x.clone() for x in sets[0]], t.zeros_like(sets[0][0]), _ws(n)
    graph, side = t.cuda.CUDAGraph(), t.cuda.Stream()
    with t.cuda.graph(graph):
        qa.attn_kv4_tree(held[0], *parts, held[1], held[3], o, 2, T, 2, q_lens=held[2], ws=ws)
    for i in (0, 1, 2, 0, 2):
        for h, s in zip(held, sets[i]):
            h.copy_(s)
        o.zero_()
        j = (i + 1) % 3
        p, own = t.zeros_like(o), _ws(n)
        side.wait_stream(t.cuda.current_stream())
        graph.replay()
        with t.cuda.stream(side):
            qa.attn_kv4_tree(sets[j][0], *parts, sets[j][1], sets[j][3], p, 2, T, 2, q_lens=sets[j][2], ws=own)
        t.cuda.synchronize()
        assert t.equal(o, want[i]) and t.equal(p, want[j])


@pytest.mark.parametrize("D,T", [(64, 60), (128, 100), (64, 200), (128, 150)])
def test_queries_that_are_not_finite_stay_with_their_row(D, T):
    """A token's NaN or infinity reaches its own row only, where waves' and shares' sums are joined, too."""
    qa, t = _qa(), torch()
    case = CacheCase(34, 1, 1, D, 64, [3000], extra_pages=2000)
    parts, lens = case.device(dev), dev(np.array([3000], np.int32))
    q = t.randn((T, 2 * D), device="cuda", generator=t.Generator(device="cuda").manual_seed(7)).bfloat16()
    word = dev(O.words(O.ancestors([-1] * T)))
    n = qa.attn_kv4_tree_workspace(1, T, 2, 1, D, case.cache.table.shape[1] * 64)
    out = []
    for bad in (None, float("nan"), float("inf")):
        x, o = q.clone(), t.empty_like(q)
        if bad is not None:
            x[1, D + 7] = bad
        qa.attn_kv4_tree(x, *parts, lens, word, o, 1, T, 2, ws=_ws(n))
        out.append(o)
    mask = t.ones_like(q, dtype=t.bool)
    mask[1, D:] = False
    for o in out[1:]:
        assert not bool(o[1, D:].isfinite().any()) and bool(o[mask].isfinite().all())
        # (the other rows' references may move with their tile: within their roundings)
        assert float((o[mask].float() - out[0][mask].float()).abs().max()) <= 2.0 ** -6 * float(out[0].abs().max())


_Short = CacheCase


class _Long(_Short):
    """A table of `to` entries a stream, those behind the cache's pages of no page."""
    to = 1 << 14

    def __init__(self, *a, **kw):
        super().__init__(*a, **kw)
        at = self.cache.table
        self.cache.table = np.pad(at, ((0, 0), (0, self.to - at.shape[1])), constant_values=-1)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,Hq,H", [(17, 1, 1), (8, 4, 1), (31, 2, 2), (12, 4, 1), (16, 4, 1), (63, 1, 1)])
def test_two_sixteens_of_rows_a_wave(monkeypatch, D, T, Hq, H):
    """Few rows of a key head over very long tables (the lengths are short, so most splits are empty)."""
    import tests.test_gpu_attn_tree as m
    monkeypatch.setattr(m, "CacheCase", _Long)
    rows, lens = T * (Hq // H), [3000, T, T + 70]
    assert 3 * H * -(-rows // 16) * (_Long.to * 64 // 64) * D >= 1024 * 20 * 128 and rows > 16
    assert rows <= 48 or 3 * H * -(-rows // 16) * _Long.to >= 64 * 1024
    _tree(35, 3, T, Hq, H, D, 64, lens)
    _tree(35, 3, T, Hq, H, D, 64, lens, q_lens=[T, 0, 1], kind="bits", ws=0)
    _tree(36, 3, T, Hq, H, D, 64, [T + 500, 3, 0], kind="bits", ws=1_000_000)


def test_two_sixteens_hide_any_bytes_and_other_rows(monkeypatch):
    import tests.test_gpu_attn_tree as m
    for cls in (m, __import__(__name__, fromlist=["x"])):
        monkeypatch.setattr(cls, "CacheCase", _Long)
    for D in (64, 128):
        test_a_token_that_a_row_does_not_see_may_hold_any_bytes(D, 20, 1)
    m.test_queries_that_are_not_finite_stay_with_their_row(20)


def test_gate():
    qa, t = _qa(), torch()
    for T, H in ((60, 1), (100, 8), (65, 32)):
        case = CacheCase(33, 1, H, 64, 64, [300], extra_pages=2500 if H == 1 else 300)
        q = t.ones((T, H * 64), dtype=t.bfloat16, device="cuda")
        o = t.full_like(q, 7.0)
        word = dev(O.words(np.ones((T, T), bool)))
        n = qa.attn_kv4_tree_workspace(1, T, H, H, 64, case.cache.table.shape[1] * 64)
        with qa.gate(t.zeros(1, dtype=t.uint8, device="cuda"), 1):
            qa.attn_kv4_tree(q, *case.device(dev), dev(np.array([300], np.int32)), word, o, 1, T, H, ws=_ws(n))
        assert (o == 7.0).all()
