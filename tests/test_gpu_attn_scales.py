"""Tensor scales of a key/value cache that are negative, zero or not finite."""
import numpy as np
import pytest

from oracle import attn as A
from tests._attn import U_F16, CacheCase, attn_tol, bits, rng, val
from tests._gpu import dev, host, torch

pytestmark = pytest.mark.gpu

LENS = [300, 40, 0]


def _qa():
    import mixed_precision_quantized_act_amd as qa
    return qa


def _run(case, q, ts, Lq, Hq, D, causal, scale=None):
    qa, t = _qa(), torch()
    parts = case.device(dev)
    parts[4], parts[5] = (dev(np.array([x], np.float32)) for x in ts)
    o = t.full((3 * Lq, Hq * D), 7.0, dtype=t.bfloat16, device="cuda")
    n = qa.attn_kv4_workspace(3, Lq, Hq, case.H, D, case.cache.table.shape[1] * case.page)
    ws = t.full((max(n, 16),), 0xFF, dtype=t.uint8, device="cuda")
    qa.attn_kv4(dev(q.reshape(3 * Lq, Hq * D)).view(t.bfloat16), *parts, dev(np.array(LENS, np.int32)), o, 3, Lq, Hq,
                causal=causal, scale=scale, ws=ws)
    t.cuda.synchronize()
    return val(host(o)).reshape(3, Lq, Hq, D)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Lq", [1, 20, 130])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("signs", [(-1, 1), (1, -1), (-1, -1), (0, 1), (1, 0)])
def test_any_finite_scale(D, Lq, causal, signs):
    Hq = 4
    case = CacheCase(37, 3, 2, D, 16, [max(n, 1) for n in LENS])
    g = rng(702, D, Lq)
    q = bits(g.standard_normal((3, Lq, Hq, D)))
    ts = [float(s * x) for s, x in zip(signs, case.ts)]
    case.cache.ts = np.array(ts)
    case.lens = LENS
    o, spread, logit = case.expect(q, [Lq] * 3, causal, D ** -0.5)
    got = _run(case, q, ts, Lq, Hq, D, causal)
    tol = attn_tol(o, spread, logit, D, max(LENS), U_F16, 6 * 448 * abs(ts[1]))
    assert np.all(np.abs(got - o) <= tol)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Lq", [1, 20, 130])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_key_scale_that_is_not_finite(D, Lq, bad):
    """Its logits are no numbers: NaN for every row that sees a key, zeros for
    the others (streams without keys, rows before a stream's first position)."""
    case = CacheCase(38, 3, 2, D, 16, [max(n, 1) for n in LENS])
    q = bits(rng(703, D, Lq).standard_normal((3, Lq, 4, D)))
    got = _run(case, q, (bad, float(case.ts[1])), Lq, 4, D, True)
    for b, n in enumerate(LENS):
        sees = n - (Lq - 1 - np.arange(Lq)) > 0
        assert np.isnan(got[b][sees]).all() and np.all(got[b][~sees] == 0)


@pytest.mark.parametrize("Lq", [1, 20, 130])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_value_scale_that_is_not_finite(Lq, bad):
    case = CacheCase(39, 3, 2, 64, 16, [max(n, 1) for n in LENS])
    q = bits(rng(704, Lq).standard_normal((3, Lq, 4, 64)))
    got = _run(case, q, (float(case.ts[0]), bad), Lq, 4, 64, True)
    for b, n in enumerate(LENS):
        sees = n - (Lq - 1 - np.arange(Lq)) > 0
        assert not np.isfinite(got[b][sees]).any() and np.all(got[b][~sees] == 0)


@pytest.mark.parametrize("Lq", [1, 20, 130])
def test_logits_beyond_float32_leave_rows_without_keys_alone(Lq):
    """A scale that takes the logits past float32: whatever the rows that see
    keys hold, the others are zeros."""
    case = CacheCase(40, 3, 2, 64, 16, [max(n, 1) for n in LENS])
    q = bits(rng(705, Lq).standard_normal((3, Lq, 4, 64)) * 2.0 ** 100)
    got = _run(case, q, (1e30, float(case.ts[1])), Lq, 4, 64, True, scale=1e20)
    for b, n in enumerate(LENS):
        sees = n - (Lq - 1 - np.arange(Lq)) > 0
        assert np.all(got[b][~sees] == 0)


@pytest.mark.parametrize("Lq", [1, 20, 300])
@pytest.mark.parametrize("Lk", [100, 700])
@pytest.mark.parametrize("scale", [3e38, 1e-38])
def test_states_with_the_largest_and_smallest_scale(Lq, Lk, scale):
    """Sequences that see nothing give zeros; with logits near zero the others give the average of what they see."""
    qa, t = _qa(), torch()
    g = rng(706, Lq, Lk)
    q, k, v = (bits(g.standard_normal((3 * n, 128))) for n in (Lq, Lk, Lk))
    m = np.ones((3, Lk), np.uint8)
    m[1] = 0
    o = t.full((3 * Lq, 128), 7.0, dtype=t.bfloat16, device="cuda")
    qd, kd, vd = (dev(x).view(t.bfloat16) for x in (q, k, v))
    ws = t.full((max(qa.attn_cross_workspace(3, Lq, Lk, 2, 2, 64), 16),), 0xFF, dtype=t.uint8, device="cuda")
    qa.attn_cross(qd, kd, vd, o, 3, Lq, Lk, 2, 2, 64, mask=dev(m), k_lens=dev(np.array([Lk, Lk, 60], np.int32)),
                  scale=scale, ws=ws)
    t.cuda.synchronize()
    got = val(host(o)).reshape(3, Lq, 2, 64)
    assert np.all(got[1] == 0)
    if scale < 1:
        for b, n in ((0, Lk), (2, 60)):
            vv = val(v).reshape(3, Lk, 2, 64)[b, :n]
            want, spread = vv.mean(0), np.abs(vv).mean(0)
            assert np.all(np.abs(got[b] - want) <= attn_tol(want, spread, 0.0, 64, Lk, 2.0 ** -8, 0.0))
