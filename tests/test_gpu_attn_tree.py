"""attn_kv4_tree against softmax attention in float64."""
import numpy as np
import pytest

from oracle import attn as A
from oracle import drafts as O
from tests._attn import U_F16, CacheCase, attn_tol, bits, rng, val
from tests._gpu import dev, host, torch

pytestmark = pytest.mark.gpu


def _qa():
    import mixed_precision_quantized_act_amd as qa
    return qa


def _trees(g, B, T, kind):
    """bool [B, T, T]: random trees, or any bits at all (empty rows among them)."""
    if kind == "bits":
        s = g.random((B, T, T)) < 0.3
        s[:, T // 2] = False
        return s
    return np.stack([O.ancestors([-1] + [int(g.integers(-1, i)) for i in range(1, T)]) for _ in range(B)])


def _ws(n):
    t = torch()
    return t.full((max(n, 16),), 0xFF, dtype=t.uint8, device="cuda")      # NaN, whatever is read of it


def _tree(seed, B, T, Hq, H, D, page, lens, q_lens=None, kind="tree", shared=False, ws="full", pad=0, cap=None,
          gain=1.0, scale=None, **kw):
    qa, t = _qa(), torch()
    g = rng(711, seed, B, T, Hq, D)
    case = CacheCase(seed, B, H, D, page, [max(1, n) for n in lens], **kw)
    q = bits(g.standard_normal((B, T, Hq, D)) * gain)
    ql = [T] * B if q_lens is None else q_lens
    seen = _trees(g, 1 if shared else B, T, kind)
    word = O.words(seen)
    if T % 64:                       # bits past the last token mean nothing
        word[..., -1] |= np.int64(-1) << np.int64(T % 64)
    w, cols = Hq * D, case.cache.table.shape[1] * page
    qd = t.full((B * T, w + pad), float("nan"), dtype=t.bfloat16, device="cuda")
    qd[:, :w] = dev(q.reshape(B * T, w)).view(t.bfloat16)
    for b in range(B):               # rows behind a stream's tokens are not read
        qd[b * T + ql[b]:(b + 1) * T] = float("nan")
    od = t.full((B * T + 1, w + pad), 7.0, dtype=t.bfloat16, device="cuda")
    nws = qa.attn_kv4_tree_workspace(B, T, Hq, H, D, cols) if ws == "full" else ws
    ln = np.asarray(lens, np.int32) if cap is None else np.full(B, cap, np.int32)
    qa.attn_kv4_tree(qd, *case.device(dev), dev(ln), dev(word[0] if shared else word), od, B, T, Hq,
                     q_lens=None if q_lens is None else dev(np.asarray(q_lens, np.int32)), scale=scale,
                     ws=_ws(nws) if nws else None)
    t.cuda.synchronize()
    oh = val(host(od))
    got = oh[:B * T, :w].reshape(B, T, Hq, D)
    sc = D ** -0.5 if scale is None else scale
    for b in range(B):
        assert np.all(got[b, ql[b]:] == 7.0)
        n, m = min(lens[b], cols), ql[b]
        if not m:
            continue
        k, v, has = case.cache.values(b, n)
        s = O.tree_sees(seen[0 if shared else b], m, n) & has[None]
        qv = val(q[b, :m])
        o, spread = A.attention(qv, k, v, s, sc)
        logit = np.abs(qv).sum(-1).max() * np.abs(k).max() * sc if n else 0.0
        tol = attn_tol(o, spread, logit, D, max(n, 1), U_F16, 6 * 448 * float(case.ts[1]))
        bad = ~(np.abs(got[b, :m] - o) <= tol)
        assert not bad.any(), (b, np.argwhere(bad)[:4], got[b, :m][bad][:4], o[bad][:4], tol[bad][:4])
        assert np.all(got[b, :m][~s.any(1)] == 0)
    assert np.all(oh[B * T] == 7.0) and np.all(oh[:, w:] == 7.0)
    return got


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,H", [(1, 1), (3, 3), (4, 1), (6, 2), (16, 1), (20, 1)])
@pytest.mark.parametrize("T", [1, 2, 5])
def test_heads(D, Hq, H, T):
    _tree(1, 3, T, Hq, H, D, 16, [5, 17 + T, 200])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [3, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 200, 257])
@pytest.mark.parametrize("kind", ["tree", "bits"])
def test_tokens(D, T, kind):
    _tree(2, 2, T, 2, 1, D, 32, [T, T + 70], kind=kind)
    _tree(2, 1, T, 6, 2, D, 64, [T + 301], kind=kind, pad=8)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("prefix", [0, 1, 15, 16, 17, 47, 48, 49, 63, 64, 65, 127, 128, 129])
def test_where_the_tokens_begin(D, page, prefix):
    """The tokens' bits begin at any place in a tile of keys, and end in any."""
    for T in (9, 70):
        _tree(3, 2, T, 2, 1, D, page, [T + prefix, T + prefix + 1])


def test_ragged_tokens_and_one_tree_for_all():
    _tree(4, 5, 9, 4, 2, 64, 16, [30, 9, 1, 100, 64], q_lens=[9, 0, 1, 1, 5])
    _tree(4, 3, 150, 2, 1, 128, 64, [150, 700, 90], q_lens=[150, 1, 77], shared=True)
    _tree(4, 4, 150, 2, 1, 64, 64, [150, 700, 90, 200], q_lens=[0, 129, 64, 65], kind="bits")
    _tree(4, 3, 13, 4, 4, 128, 16, [200, 13, 14], shared=True, kind="bits")


def test_rows_without_sight():
    """Streams without positions, more tokens than positions, rows of no bits before an empty prefix."""
    got = _tree(5, 3, 12, 4, 2, 64, 16, [5, 0, 12], kind="bits")
    assert np.all(got[1] == 0)
    _tree(5, 3, 12, 4, 2, 64, 16, [5, 0, 12])
    _tree(5, 3, 70, 4, 2, 128, 16, [20, 70, 0], kind="bits")
    _tree(5, 3, 70, 4, 2, 64, 16, [64, 65, 1])


def test_pages_without_a_place():
    bad = ((0, 1, -1), (0, 2, 10 ** 8), (1, 0, -2 ** 31), (1, 6, -5))
    for T in (4, 40, 100):
        _tree(6, 2, T, 4, 2, 64, 16, [120, 110], bad=bad)
        _tree(6, 2, T, 2, 2, 128, 16, [120, 110], bad=bad, kind="bits")
    _tree(6, 1, 3, 2, 2, 64, 16, [64], extra_pages=0, cap=10 ** 6)
    _tree(6, 1, 33, 2, 2, 64, 16, [64], extra_pages=0, cap=2 ** 31 - 1)
    _tree(6, 1, 5, 2, 2, 64, 16, [16], extra_pages=0, bad=((0, 0, -1),))


@pytest.mark.parametrize("T,Hq,H", [(5, 4, 1), (40, 2, 1), (90, 3, 3), (33, 8, 2)])
def test_any_workspace(T, Hq, H):
    for D in (64, 128):
        for ws in ("full", 0, 100_000):
            _tree(7, 2, T, Hq, H, D, 64, [3000, 37 + T], ws=ws)


@pytest.mark.parametrize("gain,scale", [(60.0, None), (1e-3, None), (1.0, 3.0), (1.0, 1e-6)])
def test_sizes_of_queries_and_scale(gain, scale):
    for T in (6, 40, 130):
        _tree(8, 2, T, 4, 2, 64, 16, [200, T], gain=gain, scale=scale)
        _tree(8, 2, T, 2, 2, 128, 16, [200, T], gain=gain, scale=scale, kind="bits")


def test_the_largest_tree():
    _tree(9, 1, 1024, 1, 1, 64, 64, [1500])
    _tree(9, 2, 1000, 2, 1, 128, 32, [1000, 1111], q_lens=[1000, 961], kind="bits")


@pytest.mark.parametrize("T", [7, 70])
@pytest.mark.parametrize("D", [64, 128])
def test_a_chain_is_causal(T, D):
    """Every token the child of the one before it: the same bits as attn_kv4's causal rows."""
    qa, t = _qa(), torch()
    case = CacheCase(12, 2, 2, D, 16, [300, T])
    parts, lens = case.device(dev), dev(np.array([300, T], np.int32))
    q = t.randn((2 * T, 4 * D), device="cuda").bfloat16()
    n = qa.attn_kv4_workspace(2, T, 4, 2, D, case.cache.table.shape[1] * 16)
    word = dev(O.words(O.ancestors(np.arange(T) - 1)))
    o, p = t.empty_like(q), t.empty_like(q)
    qa.attn_kv4(q, *parts, lens, o, 2, T, 4, ws=_ws(n))
    qa.attn_kv4_tree(q, *parts, lens, word, p, 2, T, 4, ws=_ws(n))
    # (both within their own roundings of the same value: two of the output's, the weights' 2^-11 each)
    assert float((o.float() - p.float()).abs().max()) <= (2 * 2.0 ** -8 + 2 * 2.0 ** -11) * float(o.abs().max()) * 2


def test_repeat_and_gate():
    qa, t = _qa(), torch()
    for T in (5, 80):
        a = _tree(10, 2, T, 4, 2, 64, 16, [700, 100])
        assert np.array_equal(a, _tree(10, 2, T, 4, 2, 64, 16, [700, 100]))
        case = CacheCase(10, 1, 2, 64, 16, [300])
        q = t.ones((T, 128), dtype=t.bfloat16, device="cuda")
        o = t.full_like(q, 7.0)
        word = dev(O.words(np.ones((T, T), bool)))
        with qa.gate(t.zeros(1, dtype=t.uint8, device="cuda"), 1):
            qa.attn_kv4_tree(q, *case.device(dev), dev(np.array([300], np.int32)), word, o, 1, T, 2, ws=_ws(1 << 20))
        assert (o == 7.0).all()


@pytest.mark.parametrize("T", [3, 20, 130])
def test_queries_that_are_not_finite_stay_with_their_row(T):
    """A token's NaN or infinity reaches its own row only."""
    qa, t = _qa(), torch()
    case = CacheCase(13, 1, 1, 64, 16, [400])
    parts, lens = case.device(dev), dev(np.array([400], np.int32))
    q = t.randn((T, 2 * 64), device="cuda", generator=t.Generator(device="cuda").manual_seed(5)).bfloat16()
    word = dev(O.words(O.ancestors([-1] * T)))
    n = qa.attn_kv4_tree_workspace(1, T, 2, 1, 64, 4096)
    out = []
    for bad in (None, float("nan"), float("inf")):
        x, o = q.clone(), t.empty_like(q)
        if bad is not None:
            x[1, 64 + 7] = bad
        qa.attn_kv4_tree(x, *parts, lens, word, o, 1, T, 2, ws=_ws(n))
        out.append(o)
    for o in out[1:]:
        assert not bool(o[1, 64:].isfinite().any())
        mask = t.ones_like(o, dtype=t.bool)
        mask[1, 64:] = False
        assert bool(o[mask].isfinite().all())
        # (the other rows' references may move with their tile: within their roundings)
        assert float((o[mask].float() - out[0][mask].float()).abs().max()) <= 2.0 ** -6 * float(out[0].abs().max())


@pytest.mark.parametrize("T", [6, 90])
def test_captured_and_replayed(T):
    qa, t = _qa(), torch()
    g = rng(712, T)
    case = CacheCase(14, 2, 2, 64, 16, [500, 300])
    parts = case.device(dev)
    n = qa.attn_kv4_tree_workspace(2, T, 4, 2, 64, case.cache.table.shape[1] * 16)
    sets = [(t.randn((2 * T, 256), device="cuda").bfloat16(), dev(np.array(ln, np.int32)), dev(np.array(m, np.int32)),
             dev(O.words(_trees(g, 2, T, "tree")))) for ln, m in (([500, 300], [T, T]), ([T, 200], [T, 1]), ([90, 91], [3, T]))]
    want = []
    for q, ln, m, word in sets:
        o = t.zeros_like(q)
        qa.attn_kv4_tree(q, *parts, ln, word, o, 2, T, 4, q_lens=m, ws=_ws(n))
        want.append(o)
    held, o, ws = [x.clone() for x in sets[0]], t.zeros_like(sets[0][0]), _ws(n)
    graph = t.cuda.CUDAGraph()
    side = t.cuda.Stream()
    with t.cuda.graph(graph):
        qa.attn_kv4_tree(held[0], *parts, held[1], held[3], o, 2, T, 4, q_lens=held[2], ws=ws)
    for i in (0, 1, 2, 0, 2):
        for h, s in zip(held, sets[i]):
            h.copy_(s)
        o.zero_()
        graph.replay()
        assert t.equal(o, want[i])
        j = (i + 1) % 3
        p, own = t.zeros_like(o), _ws(n)
        side.wait_stream(t.cuda.current_stream())
        with t.cuda.stream(side):
            qa.attn_kv4_tree(sets[j][0], *parts, sets[j][1], sets[j][3], p, 2, T, 4, q_lens=sets[j][2], ws=own)
        t.cuda.synchronize()
        assert t.equal(p, want[j])
