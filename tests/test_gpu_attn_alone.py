"""Queries that are not finite beside others: every other row and head keeps
the result that it has alone, to the tolerance of its own values (not of the
largest), against float64."""
import numpy as np
import pytest

from oracle import attn as A
from tests._attn import U_BF16, U_F16, CacheCase, attn_tol, bits, rng, val
from tests._gpu import dev, host, torch

pytestmark = pytest.mark.gpu

NAN, INF, NINF = 0x7FC0, 0x7F80, 0xFF80


def _qa():
    import mixed_precision_quantized_act_amd as qa
    return qa


def _ws(n):
    t = torch()
    return t.full((max(n, 16),), 0xFF, dtype=t.uint8, device="cuda")


def _poison(q, g):
    """One element of a seventh of the (row, head) pairs, row 0 head 0 among
    them; returns which pairs."""
    Lq, H, D = q.shape
    hit = g.random((Lq, H)) < 1 / 7
    hit[0, 0] = True
    for r, h in np.argwhere(hit):
        q[r, h, g.integers(0, D)] = (NAN, INF, NINF)[g.integers(0, 3)]
    if hit.all():
        hit[-1, -1] = False
        q[-1, -1] = 0x3F80
    return hit


def _check(got, hit, q, k, v, seen, scale, D, u_p, vmax):
    clean = np.where(hit[..., None], 0.0, val(q))
    o, spread = A.attention(clean, k, v, seen, scale)
    logit = np.abs(clean).sum(-1).max() * np.abs(k).max() * scale
    tol = attn_tol(o, spread, logit, D, len(k), u_p, vmax)
    bad = ~(np.abs(got - o) <= tol) & ~hit[..., None]
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], o[bad][:4], tol[bad][:4])
    assert not np.isfinite(got[hit]).all(-1).any()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Lq", [3, 20, 70, 300])
@pytest.mark.parametrize("Lk", [100, 400, 700])
def test_states(D, Lq, Lk):
    qa, t = _qa(), torch()
    H = 2
    g = rng(805, D, Lq, Lk)
    q, k, v = (bits(g.standard_normal((n, H, D))) for n in (Lq, Lk, Lk))
    hit = _poison(q, g)
    o = t.empty((Lq, H * D), dtype=t.bfloat16, device="cuda")
    qd, kd, vd = (dev(x.reshape(len(x), -1)).view(t.bfloat16) for x in (q, k, v))
    qa.attn_cross(qd, kd, vd, o, 1, Lq, Lk, H, H, D, ws=_ws(qa.attn_cross_workspace(1, Lq, Lk, H, H, D)))
    got = val(host(o)).reshape(Lq, H, D)
    _check(got, hit, q, val(k), val(v), np.ones((Lq, Lk), bool), D ** -0.5, D, U_BF16, 0.0)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Lq", [3, 20, 70, 300])
@pytest.mark.parametrize("n", [310, 900])
@pytest.mark.parametrize("causal", [True, False])
def test_cache(D, Lq, n, causal):
    qa, t = _qa(), torch()
    H = 2
    case = CacheCase(43, 1, H, D, 16, [n])
    g = rng(806, D, Lq, n)
    q = bits(g.standard_normal((Lq, H, D)))
    hit = _poison(q, g)
    o = t.empty((Lq, H * D), dtype=t.bfloat16, device="cuda")
    ws = _ws(qa.attn_kv4_workspace(1, Lq, H, H, D, case.cache.table.shape[1] * 16))
    qa.attn_kv4(dev(q.reshape(Lq, H * D)).view(t.bfloat16), *case.device(dev), dev(np.array([n], np.int32)), o, 1, Lq, H,
                causal=causal, ws=ws)
    got = val(host(o)).reshape(Lq, H, D)
    k, v, has = case.cache.values(0, n)
    assert has.all()
    upto = n - (Lq - 1 - np.arange(Lq)) if causal else np.full(Lq, n)
    seen = np.arange(n)[None] < upto[:, None]
    _check(got, hit, q, k, v, seen, D ** -0.5, D, U_F16, 6 * 448 * float(case.ts[1]))
