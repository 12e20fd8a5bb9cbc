"""attn_kv4 and attn_cross where one way of working ends and the next begins,
with values that are not finite, workspaces of other sizes and calls that
share one; the entry points' refusals."""
import numpy as np
import pytest

from tests._attn import CacheCase, bits, rng
from tests._gpu import dev, host, torch
from tests.test_gpu_attn import _cross, _kv4, _ws

pytestmark = pytest.mark.gpu


def _qa():
    import mixed_precision_quantized_act_amd as qa
    return qa


# ------------------------------------------------- sizes at which ways part --

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Lk", [255, 256, 257])
@pytest.mark.parametrize("Lq,Hq,H", [(255, 1, 1), (256, 1, 1), (257, 1, 1), (128, 4, 2), (86, 3, 1)])
def test_cross_rows_and_states_around_the_few_states_kernel(D, Lk, Lq, Hq, H):
    _cross(21, 1, Lq, Lk, Hq, H, D)


@pytest.mark.parametrize("D", [64, 128])
def test_cross_few_states_of_many_sequences(D):
    _cross(22, 70, 260, 5, 2, 2, D, k_lens=[(3 * b) % 7 for b in range(70)])


@pytest.mark.parametrize("D", [64, 128])
def test_cross_few_states_shared_by_many_workgroups(D):
    _cross(23, 1, 5000, 130, 1, 1, D, pad=8)


@pytest.mark.parametrize("Lq", [1, 40, 300])
def test_cross_nothing_seen_before_the_last_states(Lq):
    """The first tiles of the states hold nothing that is seen."""
    m = np.zeros((3, 250), bool)
    m[0, 249] = m[1, 130:140] = m[2, 64:] = True
    _cross(24, 3, Lq, 250, 2, 2, 64, mask=m)
    _cross(24, 3, Lq, 250, 2, 1, 128, mask=m)


@pytest.mark.parametrize("rows", [63, 64, 65])
def test_kv4_rows_around_the_many_rows_kernel(rows):
    _kv4(25, 2, rows, 2, 2, 64, 16, [rows + 100, rows])
    _kv4(25, 2, rows, 2, 2, 128, 16, [rows + 100, rows])


@pytest.mark.parametrize("ws", ["full", 0, 200_000, 700_000])
@pytest.mark.parametrize("causal", [True, False])
def test_kv4_many_rows_split_over_workgroups(ws, causal):
    """Few tiles of rows, many keys: the keys are taken in pieces as the workspace allows."""
    _kv4(26, 1, 300, 1, 1, 64, 64, [3001], causal=causal, ws=ws)
    _kv4(26, 2, 70, 2, 1, 128, 16, [1300, 71], causal=causal, ws=ws)


@pytest.mark.parametrize("ws", ["full", 0, 300_000])
def test_cross_many_rows_split_over_workgroups(ws):
    _cross(27, 1, 300, 2600, 1, 1, 64, ws=ws)
    _cross(27, 2, 130, 1500, 2, 1, 128, k_lens=[1500, 3], ws=ws)


def test_one_stream_of_many_lengths_behind_one_table():
    """The work is laid out for the table's length, whatever the stream's own."""
    for n in (1, 64, 257, 5000):
        case_lens = [n, 5000]
        _kv4(28, 2, 1, 4, 1, 64, 64, case_lens)


# --------------------------------------------------------- growing maxima --

@pytest.mark.parametrize("order", ["up", "down", "spikes"])
@pytest.mark.parametrize("Lq", [1, 70, 300])
def test_cross_logits_in_order(order, Lq):
    """Logits that grow by 2 to 30 from state to state, that fall, and single
    ones that stand far above the rest."""
    from oracle import attn as A
    from tests._attn import U_BF16, attn_tol, val
    qa, t = _qa(), torch()
    D, Lk = 64, 700 if Lq > 1 else 300
    for Lk in (Lk, 200):
        g = rng(803, Lq, Lk)
        q = np.zeros((Lq, D))
        q[:, 0] = 1.0 + np.arange(Lq) % 3
        k = g.standard_normal((Lk, D)) * 0.01
        step = np.linspace(2.0, 30.0, Lk)
        k[:, 0] = {"up": np.cumsum(step) / 20, "down": -np.cumsum(step) / 20,
                   "spikes": np.where(np.arange(Lk) % 97 == 50, 200.0 + np.arange(Lk), 0.0)}[order]
        v = g.standard_normal((Lk, D))
        qb, kb, vb = bits(q), bits(k), bits(v)
        o = t.empty((Lq, D), dtype=t.bfloat16, device="cuda")
        as_bf = lambda a: dev(a).view(t.bfloat16)  # noqa: E731
        qa.attn_cross(as_bf(qb), as_bf(kb), as_bf(vb), o, 1, Lq, Lk, 1, 1, D, scale=1.0,
                      ws=_ws(qa.attn_cross_workspace(1, Lq, Lk, 1, 1, D)))
        got = val(host(o))[:, None]
        qv, kv, vv = val(qb)[:, None], val(kb)[:, None], val(vb)[:, None]
        want, spread = A.attention(qv, kv, vv, np.ones((Lq, Lk), bool), 1.0)
        logit = np.abs(qv).sum(-1).max() * np.abs(kv).max()
        tol = attn_tol(want, spread, logit, D, Lk, U_BF16, 0.0)
        assert np.all(np.abs(got - want) <= tol)


# ------------------------------------------------------------- not finite --

@pytest.mark.parametrize("Lq", [3, 70, 300])
@pytest.mark.parametrize("D", [64, 128])
def test_cross_a_query_that_is_not_finite_stays_alone(Lq, D):
    """Other rows keep finite results near those without it (a row beside may
    round its weights to another reference: twice the weights' half step)."""
    qa, t = _qa(), torch()
    g = t.Generator(device="cuda").manual_seed(6)
    for Lk in (100, 600):
        q = t.randn((Lq, 2 * D), generator=g, device="cuda").bfloat16()
        k, v = (t.randn((Lk, 2 * D), generator=g, device="cuda").bfloat16() for _ in range(2))
        o, o2 = t.empty_like(q), t.empty_like(q)
        ws = _ws(qa.attn_cross_workspace(1, Lq, Lk, 2, 2, D))
        qa.attn_cross(q, k, v, o, 1, Lq, Lk, 2, 2, D, ws=ws)
        q[1, 5] = float("nan")
        qa.attn_cross(q, k, v, o2, 1, Lq, Lk, 2, 2, D, ws=ws)
        assert o2[1, :D].isnan().all() and not o2[1, D:].isnan().any()
        keep = [i for i in range(Lq) if i != 1]
        # |v| <= 6 here: 2 x 2^-8 of it for the weights, 2^-8 for the outputs' own rounding, each side
        assert float((o2[keep].float() - o[keep].float()).abs().max()) <= 6 * 4 * 2.0 ** -8


@pytest.mark.parametrize("Lq", [1, 70, 300])
def test_cross_an_infinite_value_stays_in_its_element(Lq):
    qa, t = _qa(), torch()
    g = t.Generator(device="cuda").manual_seed(7)
    for Lk in (100, 600):
        q = t.randn((Lq, 128), generator=g, device="cuda").bfloat16()
        k, v = (t.randn((Lk, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
        o, o2 = t.empty_like(q), t.empty_like(q)
        ws = _ws(qa.attn_cross_workspace(1, Lq, Lk, 2, 2, 64))
        qa.attn_cross(q, k, v, o, 1, Lq, Lk, 2, 2, 64, ws=ws)
        v[Lk // 2, 70] = float("inf")
        qa.attn_cross(q, k, v, o2, 1, Lq, Lk, 2, 2, 64, ws=ws)
        rest = [i for i in range(128) if i != 70]
        assert t.equal(o[:, rest], o2[:, rest]) and not o2[:, 70].isfinite().any()


# ----------------------------------------------- workspaces, streams, graphs --

def test_calls_that_share_a_workspace():
    """Two calls one after the other on one stream give what each gives alone;
    their order and another stream change nothing."""
    qa, t = _qa(), torch()
    case = CacheCase(31, 2, 2, 64, 16, [2500, 900])
    parts = case.device(dev)
    lens = dev(np.array([2500, 900], np.int32))
    g = t.Generator(device="cuda").manual_seed(8)
    k, v = (t.randn((2 * 1500, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
    L = case.cache.table.shape[1] * 16
    calls = []
    for Lq in (1, 90):
        q = t.randn((2 * Lq, 4 * 64), generator=g, device="cuda").bfloat16()
        calls.append((qa.attn_kv4_workspace(2, Lq, 4, 2, 64, L), q, lambda q, o, w, Lq=Lq: qa.attn_kv4(
            q, *parts, lens, o, 2, Lq, 4, ws=w)))
        calls.append((qa.attn_cross_workspace(2, Lq, 1500, 4, 2, 64), q, lambda q, o, w, Lq=Lq: qa.attn_cross(
            q, k, v, o, 2, Lq, 1500, 4, 2, 64, ws=w)))
    alone = []
    for n, q, f in calls:
        o = t.empty_like(q)
        f(q, o, _ws(n))
        t.cuda.synchronize()
        alone.append(o)
    side = t.cuda.Stream()
    for stream in (t.cuda.current_stream(), side):
        side.wait_stream(t.cuda.current_stream())
        with t.cuda.stream(stream):
            shared = _ws(max(n for n, _, _ in calls))
            outs = [t.empty_like(q) for _, q, _ in calls]
            for _ in range(3):
                for (_, q, f), o in zip(calls, outs):
                    f(q, o, shared)
                for (_, q, f), o in list(zip(calls, outs))[::-1]:
                    f(q, o, shared)
        t.cuda.synchronize()
        assert all(t.equal(a, o) for a, o in zip(alone, outs))


# --------------------------------------------------------------- refusals --

def test_tensors_that_are_refused():
    qa, t = _qa(), torch()
    case = CacheCase(32, 1, 2, 64, 16, [40])
    parts = case.device(dev)
    lens = dev(np.array([40], np.int32))
    q = t.zeros((1, 128), dtype=t.bfloat16, device="cuda")
    o = t.full_like(q, 7.0)
    kv = t.zeros((30, 128), dtype=t.bfloat16, device="cuda")

    def kv4(**c):
        a = dict(q=q, lens=lens, o=o, B=1, Hq=2, ws=None)
        a.update(c)
        qa.attn_kv4(a["q"], *parts, a["lens"], a["o"], a["B"], 1, a["Hq"], ws=a["ws"])

    def cross(**c):
        a = dict(q=q, k=kv, v=kv, o=o, k_lens=None, mask=None, ws=None)
        a.update(c)
        qa.attn_cross(a["q"], a["k"], a["v"], a["o"], 1, 1, 30, 2, 2, 64, k_lens=a["k_lens"], mask=a["mask"],
                      ws=a["ws"])

    kv4(), cross()
    t.cuda.synchronize()
    o.fill_(7.0)
    wrong = [
        lambda: kv4(q=q.cpu()), lambda: kv4(o=o.float()), lambda: kv4(q=q[:, :64]), lambda: kv4(q=q.t()),
        lambda: kv4(lens=lens.long()), lambda: kv4(lens=lens.cpu()), lambda: kv4(lens=lens[:0]),
        lambda: kv4(B=2), lambda: kv4(ws=t.zeros(8, device="cuda")),
        lambda: kv4(Hq=4),
        lambda: cross(k=kv.half()), lambda: cross(v=kv[:20]), lambda: cross(k=kv.cpu()),
        lambda: cross(mask=t.ones((1, 29), dtype=t.bool, device="cuda")),
        lambda: cross(mask=t.ones((1, 30), dtype=t.int32, device="cuda")),
        lambda: cross(mask=t.ones((30, 2), dtype=t.bool, device="cuda")[:, 0][None]),
        lambda: cross(k_lens=t.ones(1, device="cuda")),
        lambda: cross(q=t.zeros((1, 256), dtype=t.bfloat16, device="cuda")[:, ::2]),
    ]
    for i, f in enumerate(wrong):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was not refused")
    for i in range(7):                # every part of the cache
        bad = [parts[i].cpu(), parts[i].float() if i not in (4, 5) else parts[i].double()]
        if i in (0, 1, 2, 3):
            bad += [parts[i][:, :, ::2], parts[i][:-1]]
        for p in bad:
            cache = parts[:i] + [p] + parts[i + 1:]
            with pytest.raises(ValueError):
                qa.attn_kv4(q, *cache, lens, o, 1, 1, 2)
            with pytest.raises(ValueError):
                qa.kv4_append(kv[:1], kv[1:2], *cache, lens, 1, 1)
            with pytest.raises(ValueError):
                qa.kv4_read(o, t.empty_like(o), *cache, lens, 1, 1)
    with pytest.raises(qa.QactError):
        qa.attn_kv4(q, *parts, lens, o, 1, 1, 2, scale=float("nan"))
    with pytest.raises(qa.QactError):
        qa.attn_cross(q, kv, kv, q, 1, 1, 30, 2, 2, 64, ws=q.view(t.uint8)[0])
    t.cuda.synchronize()
    assert (o == 7.0).all()


def test_linear_and_norm_tensors_that_are_refused():
    qa, t = _qa(), torch()
    x, y = (t.zeros((3, n), dtype=t.bfloat16, device="cuda") for n in (64, 32))
    wq, ws = (t.zeros((32, n), dtype=t.uint8, device="cuda") for n in (32, 4))
    ts, b = t.ones(1, device="cuda"), t.zeros(32, dtype=t.bfloat16, device="cuda")

    def rows(**c):
        a = dict(x=x, w_q=wq, w_s=ws, w_ts=ts, y=y, bias=b)
        a.update(c)
        qa.qlinear_bf16(a["x"], a["w_q"], a["w_s"], a["w_ts"], a["y"], 3, 32, 64, bias=a["bias"])

    cos = t.ones((3, 32), device="cuda")

    def norm(**c):
        a = dict(q=x, q_out=t.empty_like(x), cos=cos, sin=cos.clone(), pos=None, q_w=None)
        a.update(c)
        qa.qk_norm_rope(a["q"], None, a["q_out"], None, 3, 1, 0, 64, q_w=a["q_w"], rope=qa.ROPE_PAIRS, cos=a["cos"],
                        sin=a["sin"], pos=a["pos"])

    rows(), norm()
    pos = t.zeros(2, dtype=t.int32, device="cuda")
    wrong = [
        lambda: rows(x=x[:2]), lambda: rows(x=x[:, :32]), lambda: rows(x=x.float()), lambda: rows(x=x.cpu()),
        lambda: rows(w_q=wq[:31]), lambda: rows(w_q=wq.t()), lambda: rows(w_s=ws[:, :3]), lambda: rows(w_s=ws.cpu()),
        lambda: rows(w_ts=ts[:0]), lambda: rows(w_ts=ts.double()), lambda: rows(bias=b[:31]),
        lambda: rows(y=y[:2]), lambda: rows(y=y[:, :31]), lambda: rows(y=y.float()),
        lambda: norm(q=x[:2]), lambda: norm(q_out=x[:, :32]), lambda: norm(cos=cos[:2]), lambda: norm(cos=cos.half()),
        lambda: norm(cos=t.ones((3, 64), device="cuda"), sin=t.ones((3, 64), device="cuda")),
        lambda: norm(pos=pos), lambda: norm(pos=pos.long()), lambda: norm(q_w=b),
    ]
    for i, f in enumerate(wrong):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was not refused")


@pytest.mark.parametrize("Lk", [257, 320, 449, 511, 512, 513])
@pytest.mark.parametrize("Lq,Hq,H", [(256, 1, 1), (700, 2, 1)])
def test_cross_more_of_few_states(Lk, Lq, Hq, H):
    m = rng(804, Lk).random((2, Lk)) < 0.7
    m[0, 130:] = False
    _cross(29, 2, Lq, Lk, Hq, H, 64)
    _cross(29, 2, Lq, Lk, Hq, H, 64, mask=m, k_lens=[Lk, Lk - 100])


@pytest.mark.parametrize("Lq", [1, 5])
@pytest.mark.parametrize("D", [64, 128])
def test_kv4_short_streams_behind_a_large_table(Lq, D):
    """Streams of 5 to 3000 tokens of a table for 100000: each takes the splits that its own length is worth."""
    _kv4(33, 4, Lq, 4, 2, D, 64, [5, 3000, 257, 700], extra_pages=1500, bad=[(0, 3, -1)])


@pytest.mark.parametrize("Lq", [2, 70, 300])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_kv4_a_query_that_is_not_finite_stays_alone(Lq, bad):
    """Other rows keep finite results near those without it (as above; |v| <= 6 x 448 x 6 / 2688 at most,
    fp16 weights: 2 x 2^-11 of it, 2^-8 for the outputs' own rounding, each side)."""
    qa, t = _qa(), torch()
    case = CacheCase(34, 1, 2, 64, 16, [900])
    parts = case.device(dev)
    lens = dev(np.array([900], np.int32))
    g = t.Generator(device="cuda").manual_seed(12)
    q = t.randn((Lq, 128), generator=g, device="cuda").bfloat16()
    o, o2 = t.empty_like(q), t.empty_like(q)
    ws = _ws(qa.attn_kv4_workspace(1, Lq, 2, 2, 64, case.cache.table.shape[1] * 16))
    qa.attn_kv4(q, *parts, lens, o, 1, Lq, 2, causal=False, ws=ws)
    q[1, 9] = bad
    qa.attn_kv4(q, *parts, lens, o2, 1, Lq, 2, causal=False, ws=ws)
    assert not o2[1, 64:].isnan().any() and not o2[1, :64].isfinite().all()
    keep = [i for i in range(Lq) if i != 1]
    assert float((o2[keep].float() - o[keep].float()).abs().max()) <= 6 * (4 * 2.0 ** -11 + 2 * 2.0 ** -8)
    assert t.equal(o2[1, 64:], o[1, 64:]) or Lq > 2


@pytest.mark.parametrize("Lq,lens", [(1, [3000, 20]), (100, [3000, 150]), (300, [5000, 300])])
def test_kv4_the_same_bits_every_time(Lq, lens):
    a = _kv4(35, 2, Lq, 2, 1, 64, 64, lens)
    for _ in range(3):
        assert np.array_equal(a, _kv4(35, 2, Lq, 2, 1, 64, 64, lens))
