"""Group scales of a tree's values that are NaN or negative: what they make of the rows that see them, on every way
that attn_kv4_tree takes, against float64."""
import numpy as np
import pytest

from oracle import attn as A
from oracle import drafts as O
from tests._attn import U_F16, CacheCase, attn_tol, bits, rng, val
from tests._gpu import dev, host, torch
from tests.test_gpu_attn_tree import _qa, _trees, _ws
from tests.test_gpu_attn_tree_cuts import _Long

pytestmark = pytest.mark.gpu


def _run(D, B, T, Hq, H, page, lens, odd, kind, ws="full", cls=CacheCase, q_lens=None, **kw):
    """odd(cache scales [tokens, H, D / 16] of stream b, tokens in front of the drafted ones) changes them."""
    qa, t = _qa(), torch()
    g = rng(741, D, B, T, Hq)
    case = cls(41, B, H, D, page, lens, **kw)
    ql = [T] * B if q_lens is None else q_lens
    for b, n in enumerate(lens):
        at = [case.cache.slot(b, j) for j in range(n)]
        s = np.stack([case.cache.v_s[p, :, i] for p, i in at])
        odd(g, b, s, n - ql[b])
        for (p, i), x in zip(at, s):
            case.cache.v_s[p, :, i] = x
    q, seen = bits(g.standard_normal((B, T, Hq, D))), _trees(g, B, T, kind)
    w, cols = Hq * D, case.cache.table.shape[1] * page
    o = t.full((B * T, w), 7.0, dtype=t.bfloat16, device="cuda")
    n = qa.attn_kv4_tree_workspace(B, T, Hq, H, D, cols) if ws == "full" else ws
    qa.attn_kv4_tree(dev(q.reshape(B * T, w)).view(t.bfloat16), *case.device(dev), dev(np.asarray(lens, np.int32)),
                     dev(O.words(seen)), o, B, T, Hq, q_lens=dev(np.asarray(ql, np.int32)), ws=_ws(n) if n else None)
    t.cuda.synchronize()
    got = val(host(o)).reshape(B, T, Hq, D)
    for b in range(B):
        n, m = lens[b], ql[b]
        assert np.all(got[b, m:] == 7.0)
        if not m:
            continue
        k, v, _ = case.cache.values(b, n)
        s, qv, nan = O.tree_sees(seen[b], m, n), val(q[b, :m]), np.isnan(v)
        want, spread = A.attention(qv, k, np.where(nan, 0.0, v), s, D ** -0.5)
        hit = np.einsum("tn,nhd->thd", s.astype(float), nan.astype(float)) > 0          # a row's head, element by element
        hit = np.repeat(hit, Hq // H, axis=1)
        logit = np.abs(qv).sum(-1).max() * np.abs(k).max() * D ** -0.5
        tol = attn_tol(want, spread, logit, D, n, U_F16, 6 * 448 * float(case.ts[1]))
        x = got[b, :m]
        assert np.array_equal(np.isnan(x), hit), (b, np.argwhere(np.isnan(x) != hit)[:4])
        assert np.all(np.abs(x - want)[~hit] <= tol[~hit])


def _nan_drafted(g, b, s, first):
    """One drafted token's group, all groups of another's last head."""
    if len(s) - first > 2:
        s[first + 1, 0, b % s.shape[2]] = 0x7F
        s[first + 2, -1] = 0xFF


def _nan_anywhere(g, b, s, first):
    _nan_drafted(g, b, s, first)
    if b == 1 and first > 1:
        s[first - 1, 0, 1] = 0xFF
        s[0, 0, 2] = 0x7F


def _negative(g, b, s, first):
    s[g.random(s.shape) < 0.3] |= 0x80


def _both(g, b, s, first):
    _negative(g, b, s, first)
    _nan_anywhere(g, b, s, first)


ODD = {"drafted": _nan_drafted, "anywhere": _nan_anywhere, "negative": _negative, "both": _both}


@pytest.mark.parametrize("odd", list(ODD))
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,Hq,H", [(3, 1, 1), (9, 4, 2), (16, 2, 2), (40, 1, 1)])
def test_few_rows(D, T, Hq, H, odd):
    for kind in ("tree", "bits"):
        for ws in ("full", 0):
            _run(D, 2, T, Hq, H, 16, [T + 71, T + 300], ODD[odd], kind, ws)


@pytest.mark.parametrize("odd", list(ODD))
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,Hq,H", [(20, 1, 1), (12, 4, 1)])
def test_few_rows_two_sixteens_a_wave(D, T, Hq, H, odd):
    _run(D, 3, T, Hq, H, 64, [T + 500, T + 71, T], ODD[odd], "tree", cls=_Long)
    _run(D, 3, T, Hq, H, 64, [T + 500, T + 71, T], ODD[odd], "bits", ws=0, cls=_Long, q_lens=[T, T - 1, 3])


@pytest.mark.parametrize("odd", list(ODD))
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [60, 100, 128, 150, 257])
def test_many_rows(D, T, odd):
    """Shares of the list, and without a workspace whole units."""
    for ws in ("full", 0):
        _run(D, 3, T, 1, 1, 64, [T + 700, T + 71, T], ODD[odd], "tree", ws, extra_pages=800)
    _run(D, 2, T, 2, 1, 64, [T + 333, T + 64], ODD[odd], "bits", q_lens=[T, T - 9], extra_pages=1500)


@pytest.mark.parametrize("odd", list(ODD))
def test_many_rows_in_equal_pieces(odd):
    lens = [100, 900, 301, 140, 2000, 177, 164, 101]
    _run(128, 8, 100, 8, 8, 64, lens, ODD[odd], "tree", extra_pages=92)


@pytest.mark.parametrize("T", [70, 200])
def test_units_without_keys_or_rows_between(T):
    """What one unit's values hold stays with that unit: streams of none, of one, of many tokens after it."""
    lens = [T + 200, T + 3, T + 1500, T, T + 64]
    _run(64, 5, T, 2, 2, 32, lens, _nan_anywhere, "tree", q_lens=[T, 0, T, 1, T], extra_pages=1500)
    _run(128, 5, T, 2, 2, 32, lens, _nan_anywhere, "bits", q_lens=[T, 3, 0, T, T], extra_pages=1500)
