"""attn_kv4 and attn_cross against softmax attention in float64."""
import numpy as np
import pytest

from oracle import attn as A
from tests._attn import U_BF16, U_F16, CacheCase, attn_tol, bits, rng, val
from tests._gpu import dev, host, torch

pytestmark = pytest.mark.gpu


def _qa():
    import mixed_precision_quantized_act_amd as qa
    return qa


def _ws(n):
    t = torch()
    return t.full((max(n, 16),), 0xFF, dtype=t.uint8, device="cuda")      # NaN, whatever is read of it


def _kv4(seed, B, Lq, Hq, H, D, page, lens, q_lens=None, causal=True, scale=None, ws="full", pad=0, gain=1.0, **kw):
    qa, t = _qa(), torch()
    g = rng(701, seed, B, Lq, Hq, D)
    cap = kw.pop("cap", None)
    case = CacheCase(seed, B, H, D, page, lens, **kw)
    q = bits(g.standard_normal((B, Lq, Hq, D)) * gain)
    ql = [Lq] * B if q_lens is None else q_lens
    sc = D ** -0.5 if scale is None else scale
    o, spread, logit = case.expect(q, ql, causal, sc)
    w = Hq * D
    qd = t.full((B * Lq, w + pad), float("nan"), dtype=t.bfloat16, device="cuda")
    qd[:, :w] = dev(q.reshape(B * Lq, w)).view(t.bfloat16)
    for b in range(B):              # rows behind a stream's queries are not read
        qd[b * Lq + ql[b]:(b + 1) * Lq] = float("nan")
    od = t.full((B * Lq + 1, w + pad), 7.0, dtype=t.bfloat16, device="cuda")
    L = case.cache.table.shape[1] * page
    nws = qa.attn_kv4_workspace(B, Lq, Hq, H, D, L) if ws == "full" else ws
    parts = case.device(dev)
    ln = np.asarray(lens, np.int32) if cap is None else np.full(B, cap, np.int32)
    qa.attn_kv4(qd, *parts, dev(ln), od, B, Lq, Hq,
                q_lens=None if q_lens is None else dev(np.asarray(q_lens, np.int32)), causal=causal, scale=scale,
                ws=_ws(nws) if nws else None)
    t.cuda.synchronize()
    oh = val(host(od))
    got = oh[:B * Lq, :w].reshape(B, Lq, Hq, D)
    tol = attn_tol(o, spread, logit, D, max(lens), U_F16, 6 * 448 * float(case.ts[1]))
    for b in range(B):
        assert np.all(got[b, ql[b]:] == 7.0)
        a, e, tl = got[b, :ql[b]], o[b, :ql[b]], tol[b, :ql[b]]
        bad = ~(np.abs(a - e) <= tl)
        assert not bad.any(), (b, np.argwhere(bad)[:4], a[bad][:4], e[bad][:4], tl[bad][:4])
    assert np.all(oh[B * Lq] == 7.0) and np.all(oh[:, w:] == 7.0)
    return got


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,H", [(1, 1), (3, 3), (4, 1), (6, 2), (8, 1), (16, 1), (20, 1)])
def test_single_tokens(D, Hq, H):
    _kv4(1, 3, 1, Hq, H, D, 16, [1, 17, 200])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 256])
@pytest.mark.parametrize("lens", [[1, 2, 3], [15, 16, 17], [63, 64, 65], [127, 128, 129], [255, 257, 300]])
def test_lengths_around_tiles(D, page, lens):
    _kv4(2, 3, 1, 4, 2, D, page, lens)
    _kv4(2, 3, 5, 4, 2, D, page, [max(n, 5) for n in lens])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Lq", [2, 7, 16, 17, 33, 64, 65, 130, 257])
@pytest.mark.parametrize("causal", [True, False])
def test_query_rows(D, Lq, causal):
    _kv4(3, 2, Lq, 6, 2, D, 32, [Lq, Lq + 70], causal=causal)
    _kv4(3, 1, Lq, 2, 2, D, 64, [Lq + 301], causal=causal, pad=8)


def test_long_cache_split_over_workgroups():
    for ws in ("full", 0, 50_000):
        _kv4(4, 2, 1, 2, 1, 64, 64, [5000, 37], ws=ws)
        _kv4(4, 1, 9, 3, 1, 128, 16, [3001], ws=ws)


def test_streams_without_keys_and_rows_without_sight():
    _kv4(5, 4, 1, 4, 2, 64, 16, [0, 1, 0, 40])
    # more query rows than positions: the first rows see nothing and give zeros
    got = _kv4(5, 2, 12, 4, 2, 64, 16, [5, 0], causal=True)
    assert np.all(got[0, :7] == 0) and np.all(got[1] == 0) and np.all((got[0, 7:] != 0).any(-1))
    _kv4(5, 2, 70, 4, 2, 128, 16, [20, 90], causal=True)


def test_ragged_query_rows():
    _kv4(6, 5, 9, 4, 2, 64, 16, [30, 9, 0, 100, 64], q_lens=[9, 0, 3, 1, 5])
    _kv4(6, 3, 150, 2, 1, 128, 64, [150, 700, 90], q_lens=[150, 1, 77])
    _kv4(6, 3, 150, 2, 1, 64, 64, [150, 700, 90], q_lens=[0, 129, 64], causal=False)


def test_pages_without_a_place():
    """Entries that name no page hide their positions; lengths past the table are clamped to it."""
    bad = ((0, 1, -1), (0, 2, 10 ** 8), (1, 0, -2 ** 31))
    for Lq in (1, 40, 100):
        _kv4(7, 2, Lq, 4, 2, 64, 16, [120, 110], causal=False, bad=bad)
        _kv4(7, 2, Lq, 2, 2, 128, 64, [520, 301], causal=False, bad=bad)
    _kv4(8, 1, 1, 2, 2, 64, 16, [64], extra_pages=0, cap=10 ** 6)
    _kv4(8, 1, 33, 2, 2, 64, 16, [64], extra_pages=0, cap=2 ** 31 - 1)
    _kv4(8, 1, 3, 2, 2, 64, 16, [16], extra_pages=0, bad=((0, 0, -1),))      # nothing seen at all


@pytest.mark.parametrize("gain,scale", [(60.0, None), (1e-3, None), (1.0, 3.0), (1.0, 1e-6), (2.0 ** 90, 2.0 ** -92),
                                        (2.0 ** -100, 2.0 ** 98)])
def test_sizes_of_queries_and_scale(gain, scale):
    for Lq in (1, 40):
        _kv4(9, 2, Lq, 4, 2, 64, 16, [200, 77], gain=gain, scale=scale)
        _kv4(9, 2, Lq, 2, 2, 128, 16, [200, 77], gain=gain, scale=scale)


def test_kv4_repeat_gate():
    qa, t = _qa(), torch()
    a = _kv4(10, 2, 3, 4, 2, 64, 16, [700, 33])
    assert np.array_equal(a, _kv4(10, 2, 3, 4, 2, 64, 16, [700, 33]))
    case = CacheCase(10, 1, 2, 64, 16, [300])
    for Lq in (1, 80):
        q = t.ones((Lq, 128), dtype=t.bfloat16, device="cuda")
        o = t.full_like(q, 7.0)
        with qa.gate(t.zeros(1, dtype=t.uint8, device="cuda"), 1):
            qa.attn_kv4(q, *case.device(dev), dev(np.array([300], np.int32)), o, 1, Lq, 2, ws=_ws(1 << 20))
        assert (o == 7.0).all()


def test_cache_beyond_32_bit_offsets():
    """A cache part of over 4 GiB: the pages of one stream at both of its ends."""
    qa, t = _qa(), torch()
    page, H, D = 1024, 8, 128
    pages = (1 << 32) // (page * H * D // 2) + 3
    parts = qa.empty_kv4(pages, H, page, D)
    assert parts[0].numel() > 1 << 32
    ts = t.full((1,), 4.5 / 2688, device="cuda")
    table = t.tensor([[pages - 1, 0, pages - 2]], dtype=t.int32, device="cuda")
    g = t.Generator(device="cuda").manual_seed(11)
    n = 2 * page + 100
    k, v = (t.randn((n, H * D), generator=g, device="cuda").bfloat16() for _ in range(2))
    qa.kv4_append(k, v, *parts, ts, ts, table, t.zeros(1, dtype=t.int32, device="cuda"), 1, n)
    small = [p[[pages - 1, 0, pages - 2]].contiguous() for p in parts]
    near = t.tensor([[0, 1, 2]], dtype=t.int32, device="cuda")
    lens = t.tensor([n], dtype=t.int32, device="cuda")
    for Lq in (1, 100):
        q = t.randn((Lq, H * D), generator=g, device="cuda").bfloat16()
        o, o2 = t.empty_like(q), t.empty_like(q)
        ws = _ws(qa.attn_kv4_workspace(1, Lq, H, H, D, 3 * page))
        qa.attn_kv4(q, *parts, ts, ts, table, lens, o, 1, Lq, H, ws=ws)
        qa.attn_kv4(q, *small, ts, ts, near, lens, o2, 1, Lq, H, ws=ws)
        assert t.equal(o, o2) and bool(o.abs().sum() > 0)


# ------------------------------------------------------------------- cross --

def _cross(seed, B, Lq, Lk, Hq, H, D, k_lens=None, mask=None, scale=None, ws="full", pad=0, gain=1.0, poison=True,
           kv_gain=1.0):
    qa, t = _qa(), torch()
    g = rng(801, seed, B, Lq, Lk, Hq, D)
    w, wk = Hq * D, H * D
    q = bits(g.standard_normal((B, Lq, Hq, D)) * gain)
    kv = bits(g.standard_normal((B, Lk, 2, H, D)) * kv_gain)
    seen = np.ones((B, Lk), bool)
    if k_lens is not None:
        seen &= np.arange(Lk)[None] < np.asarray(k_lens)[:, None]
    if mask is not None:
        seen &= mask != 0
    if poison:                       # what is not seen: NaN, infinities, the largest values
        junk = np.array([0x7FC0, 0xFFC1, 0x7F80, 0xFF80, 0x7F7F, 0xFF7F], np.uint16)
        kv = np.where(seen[:, :, None, None, None], kv, junk[g.integers(0, 6, kv.shape)])
    sc = D ** -0.5 if scale is None else scale
    qd = t.empty((B * Lq, w + pad), dtype=t.bfloat16, device="cuda")
    qd[:, :w] = dev(q.reshape(B * Lq, w)).view(t.bfloat16)
    kvd = dev(kv.reshape(B * Lk, 2 * wk)).view(t.bfloat16)
    od = t.full((B * Lq + 1, w + pad), 7.0, dtype=t.bfloat16, device="cuda")
    nws = qa.attn_cross_workspace(B, Lq, Lk, Hq, H, D) if ws == "full" else ws
    qa.attn_cross(qd, kvd[:, :wk], kvd[:, wk:], od, B, Lq, Lk, Hq, H, D,
                  k_lens=None if k_lens is None else dev(np.asarray(k_lens, np.int32)),
                  mask=None if mask is None else dev(mask.astype(np.uint8)), scale=scale, ws=_ws(nws) if nws else None)
    t.cuda.synchronize()
    oh = val(host(od))
    got = oh[:B * Lq, :w].reshape(B, Lq, Hq, D)
    assert np.all(oh[B * Lq] == 7.0) and np.all(oh[:, w:] == 7.0)
    for b in range(B):
        s = seen[b]
        k, v = (np.where(s[:, None, None], val(kv[b, :, i]), 0.0) for i in (0, 1))
        qv = val(q[b])
        o, spread = A.attention(qv, k, v, np.broadcast_to(s, (Lq, Lk)), sc)
        logit = np.abs(qv).sum(-1).max() * np.abs(k).max(initial=0) * sc
        tol = attn_tol(o, spread, logit, D, Lk, U_BF16, 0.0)
        bad = ~(np.abs(got[b] - o) <= tol)
        assert not bad.any(), (b, np.argwhere(bad)[:4], got[b][bad][:4], o[bad][:4], tol[bad][:4])
    return got


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Lk", [1, 2, 15, 16, 31, 33, 63, 64, 65, 100, 129, 226])
@pytest.mark.parametrize("Lq", [1, 5, 40, 150])
def test_cross_lengths(D, Lk, Lq):
    _cross(1, 2, Lq, Lk, 4, 2, D)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,H", [(1, 1), (3, 3), (5, 1), (8, 2), (32, 1)])
@pytest.mark.parametrize("Lq", [1, 3, 65])
def test_cross_heads(D, Hq, H, Lq):
    _cross(2, 3, Lq, 77, Hq, H, D, k_lens=[77, 1, 40], pad=16)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Lq", [1, 33, 300])
def test_cross_lengths_and_masks(D, Lq):
    g = rng(802, D, Lq)
    m = g.random((4, 90)) < 0.5
    m[1] = False                         # a sequence that sees nothing
    m[2, :70] = False
    got = _cross(3, 4, Lq, 90, 4, 4, D, mask=m)
    assert np.all(got[1] == 0)
    got = _cross(3, 4, Lq, 90, 4, 4, D, k_lens=[90, 5, 70, 0], mask=m)
    assert np.all(got[1:] == 0)
    _cross(3, 3, Lq, 90, 4, 4, D, k_lens=[-4, 1000, 64])


def test_cross_no_states():
    for Lq in (1, 200):
        assert np.all(_cross(4, 2, Lq, 0, 2, 2, 64) == 0)


def test_cross_long_states_split_over_workgroups():
    for ws in ("full", 0, 40_000):
        _cross(5, 2, 1, 3000, 2, 1, 64, k_lens=[3000, 129], ws=ws)
        _cross(5, 1, 11, 1500, 3, 1, 128, ws=ws)


@pytest.mark.parametrize("gain,kv_gain,scale", [(60.0, 1.0, None), (1.0, 30.0, None), (1.0, 1e-3, 3.0), (1.0, 2.0 ** 60, 2.0 ** -63)])
def test_cross_sizes_of_values(gain, kv_gain, scale):
    for Lq in (1, 70):
        _cross(6, 2, Lq, 130, 2, 2, 64, gain=gain, kv_gain=kv_gain, scale=scale)
        _cross(6, 2, Lq, 130, 2, 2, 128, gain=gain, kv_gain=kv_gain, scale=scale)


def test_cross_not_finite_where_seen():
    """A NaN key that is seen reaches every row of its head, and no other head or sequence."""
    qa, t = _qa(), torch()
    g = t.Generator(device="cuda").manual_seed(5)
    for Lq in (1, 90):
        q = t.randn((2 * Lq, 128), generator=g, device="cuda").bfloat16()
        k, v = (t.randn((2 * 50, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
        k[7, 3] = float("nan")
        o = t.empty_like(q)
        qa.attn_cross(q, k, v, o, 2, Lq, 50, 2, 2, 64, ws=_ws(1 << 20))
        nan = o.isnan()
        assert nan[:Lq, :64].all() and not nan[:Lq, 64:].any() and not nan[Lq:].any()
