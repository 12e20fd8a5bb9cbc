"""attn_kv4_tree of a chain, every token the child of the one before it, and attn_kv4's causal rows: each output of both
against float64, and a tolerance that one key too many or too few exceeds."""
import numpy as np
import pytest

from oracle import attn as A
from oracle import drafts as O
from tests._attn import U_F16, CacheCase, attn_tol, bits, rng, val
from tests._gpu import dev, host, torch
from tests.test_gpu_attn_tree import _qa, _ws

pytestmark = pytest.mark.gpu


def _shifted(case, q, b, T, off, scale):
    """The causal rows of stream b with `off` keys more."""
    n = case.lens[b]
    k, v, _ = case.cache.values(b, n)
    upto = n - (T - 1 - np.arange(T)) + off
    return A.attention(val(q), k, v, np.arange(n)[None] < upto[:, None], scale)[0]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,extra", [(1, 1), (7, 1), (70, 1), (70, 1500), (140, 1500)])
def test_a_chain_is_causal(T, extra, D):
    qa, t = _qa(), torch()
    lens, Hq, H, page = [300 + T, T, 37 + T], 4, 2, 16
    case = CacheCase(51, 3, H, D, page, lens, extra_pages=extra)
    q, scale = bits(rng(771, T, D).standard_normal((3, T, Hq, D))), D ** -0.5
    want, spread, logit = case.expect(q, [T] * 3, True, scale)
    tol = attn_tol(want, spread, logit, D, max(lens), U_F16, 6 * 448 * float(case.ts[1]))
    # what a row would be that sees the key after its own, or not its own: nine rows of ten of every stream differ by
    # more than two tolerances (a key of weight p moves an output by p |v - o|, which may be little)
    for off in (1, -1):
        other = np.stack([_shifted(case, q[b], b, T, off, scale) for b in range(3)])
        rows = slice(0, T - 1) if off == 1 else slice(1, T)
        if T > 1:
            assert np.all((np.abs(other - want) > 2 * tol).any((-1, -2))[:, rows].mean(-1) > 0.9)
    parts, ln = case.device(dev), dev(np.array(lens, np.int32))
    qd = dev(q.reshape(3 * T, Hq * D)).view(t.bfloat16)
    cols = case.cache.table.shape[1] * page
    word = dev(O.words(O.ancestors(np.arange(T) - 1)))
    o, p = t.full_like(qd, 7.0), t.full_like(qd, 7.0)
    qa.attn_kv4(qd, *parts, ln, o, 3, T, Hq, causal=True, ws=_ws(qa.attn_kv4_workspace(3, T, Hq, H, D, cols)))
    qa.attn_kv4_tree(qd, *parts, ln, word, p, 3, T, Hq, ws=_ws(qa.attn_kv4_tree_workspace(3, T, Hq, H, D, cols)))
    for x in (o, p):
        got = val(host(x)).reshape(want.shape)
        bad = ~(np.abs(got - want) <= tol)
        assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], tol[bad][:4])
