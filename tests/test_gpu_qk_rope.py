"""qk_rope against its float64 definition."""
import numpy as np
import pytest

from oracle import drafts as O
from tests._attn import U_BF16, U_F32, bits, rng, val
from tests._gpu import dev, host, torch

pytestmark = pytest.mark.gpu


def _qa():
    import mixed_precision_quantized_act_amd as qa
    return qa


def _tol(y, x, scale, turns):
    """The output's rounding; before it two products of a sine or cosine with an
    element: sine and cosine to 4 last places of float32 each, times scale,
    the products and their sum (8 half steps of |scale| (|u| + |v|) in all), and
    the angle: 2 roundings of float64 over `turns` turns, the fraction rounded
    to float32 (half a turn: pi half steps, with pi's own rounding 2 pi)."""
    angle = 7.0 * U_F32 + 2 * np.pi * turns * 2.0 ** -51
    size = abs(scale) * 2 * np.abs(x).max(-1, keepdims=True)
    return U_BF16 * np.abs(y) + size * ((8 + 4) * U_F32 + angle) * (1 + U_BF16) + 1e-37


def _run(M, Hq, Hk, D, R, rope, pos=None, scale=1.0, in_place=False, pad=0, seed=0, freq=None, gain=2.0):
    qa, t = _qa(), torch()
    g = rng(511, M, Hq, Hk, D, R, rope, seed)
    nq, nk = Hq * D, Hk * D
    qkv = bits(g.standard_normal((M, nq + 2 * nk + pad)) * gain)
    freq = O.frequencies(R, 10000.0, 0, 1.0)[0] if freq is None else freq
    d = dev(qkv).view(t.bfloat16)
    q, k = d[:, :nq], d[:, nq:nq + nk]
    if in_place:
        qo, ko = q, k
    else:
        qo = t.full((M + 1, nq + 8), 7.0, dtype=t.bfloat16, device="cuda")
        ko = t.full((M + 1, nk + 16), 7.0, dtype=t.bfloat16, device="cuda")
    qa.qk_rope(q if Hq else None, k if Hk else None, qo if Hq else None, ko if Hk else None, M, Hq, Hk, D, R, dev(freq),
               rope=rope, scale=scale, pos=None if pos is None else dev(np.asarray(pos, np.int32)))
    t.cuda.synchronize()
    at = np.arange(M) if pos is None else np.asarray(pos)
    for H, o, lo in ((Hq, qo, 0), (Hk, ko, nq)):
        if not H:
            continue
        raw = qkv[:, lo:lo + H * D].reshape(M, H, D)
        x = val(raw)
        y = O.turn(x, R, rope, freq, np.float64(np.float32(scale)), at)
        turns = (np.abs(at.astype(np.float64)) * np.abs(freq).max() / (2 * np.pi) + 1)[:, None, None]
        oh = host(o)
        if not in_place:
            assert np.all(val(oh[M]) == 7.0) and np.all(val(oh[:, H * D:]) == 7.0)
        got = oh[:M, :H * D].reshape(M, H, D)
        assert np.array_equal(got[..., R:], raw[..., R:])                      # passed on, bit by bit
        assert np.array_equal(got[at < 0], raw[at < 0])
        bad = ~(np.abs(val(got) - y) <= _tol(y, x, scale, turns))
        assert not bad.any(), (np.argwhere(bad)[:4], val(got)[bad][:4], y[bad][:4])
    if in_place:                                   # the values of the projection stay as they were
        assert np.array_equal(host(d)[:, nq + nk:], qkv[:, nq + nk:])


@pytest.mark.parametrize("rope", [1, 2])
@pytest.mark.parametrize("D,R", [(16, 16), (32, 16), (32, 32), (48, 16), (64, 16), (64, 32), (64, 48), (64, 64), (80, 32),
                                 (80, 80), (96, 64), (128, 32), (128, 64), (128, 128), (144, 112), (256, 16), (256, 64),
                                 (256, 240), (256, 256)])
def test_heads_and_parts(D, R, rope):
    _run(7, 5, 2, D, R, rope, pos=[0, 1, 2, 100, 4095, -1, 70000])
    _run(3, 4, 4, D, R, rope, in_place=True, pad=24)


@pytest.mark.parametrize("rope", [1, 2])
@pytest.mark.parametrize("M,Hq,Hk", [(1, 1, 0), (1, 0, 1), (1, 64, 64), (2, 1, 1), (33, 3, 1), (100, 30, 30), (257, 32, 8),
                                     (1000, 1, 1), (513, 7, 7), (70, 200, 3), (5, 1000, 1000)])
def test_sizes(M, Hq, Hk, rope):
    _run(M, Hq, Hk, 64, 32, rope)
    _run(M, Hq, Hk, 32, 32, rope, in_place=True)


@pytest.mark.parametrize("rope", [1, 2])
def test_far_positions_and_stretches(rope):
    pos = [0, 1, 2 ** 20 + 1, 2 ** 24 + 1, 2 ** 31 - 1, -1, -2 ** 31, 131071, 10 ** 9 + 7]
    for stretch, factor in ((0, 1.0), (1, 8.0), (2, 16.0), (3, 32.0)):
        f, s = _qa().rope_freqs(64, 10000.0, stretch, factor, 4096)
        _run(len(pos), 4, 2, 128, 64, rope, pos=pos, freq=f, scale=s)
    _run(len(pos), 4, 2, 64, 64, rope, pos=pos, freq=np.linspace(-3.0, 9.0, 32), scale=-1.75)


@pytest.mark.parametrize("rope", [1, 2])
@pytest.mark.parametrize("scale,gain", [(0.0, 1.0), (1e-20, 1.0), (3e4, 1e30), (1.0, 1e-38)])
def test_sizes_of_values(rope, scale, gain):
    _run(40, 3, 1, 64, 48, rope, scale=scale, gain=gain)


def test_elements_that_are_not_finite_stay_with_their_pair():
    qa, t = _qa(), torch()
    for rope in (1, 2):
        x = t.ones((3, 2 * 64), dtype=t.bfloat16, device="cuda")
        x[1, 5], x[1, 40], x[1, 64 + 3] = float("inf"), float("nan"), float("nan")
        x[2, 5] = float("inf")
        o = t.empty_like(x)
        qa.qk_rope(x, None, o, None, 3, 2, 0, 64, 32, dev(O.frequencies(32, 100.0, 0, 1.0)[0]), rope=rope,
                   pos=dev(np.array([3, 3, -1], np.int32)))
        bad = ~o.isfinite().cpu().numpy()
        pair = {5, 4} if rope == 1 else {5, 21}
        also = {3, 2} if rope == 1 else {3, 19}
        assert set(np.flatnonzero(bad[1])) == pair | {40} | {64 + i for i in also}
        assert not bad[0].any() and np.array_equal(host(o)[2], host(x)[2])


def test_no_tokens_and_gate():
    qa, t = _qa(), torch()
    f = dev(O.frequencies(32, 100.0, 0, 1.0)[0])
    e = t.empty((0, 128), dtype=t.bfloat16, device="cuda")
    qa.qk_rope(e, e, e, e, 0, 2, 2, 64, 32, f)
    x = t.ones((9, 128), dtype=t.bfloat16, device="cuda")
    o = t.full_like(x, 7.0)
    with qa.gate(t.zeros(1, dtype=t.uint8, device="cuda"), 1):
        qa.qk_rope(x, None, o, None, 9, 2, 0, 64, 32, f)
    assert (o == 7.0).all()


def test_agrees_with_the_rotation_by_tables():
    """Whole heads, near positions: within a rounding of qk_norm_rope with float32 tables."""
    qa, t = _qa(), torch()
    M, H, D = 50, 3, 64
    f = O.frequencies(D, 10000.0, 0, 1.0)[0]
    a = np.arange(M)[:, None] * f
    x = t.randn((M, H * D), device="cuda").bfloat16()
    for rope in (1, 2):
        o, p = t.empty_like(x), t.empty_like(x)
        qa.qk_rope(x, None, o, None, M, H, 0, D, D, dev(f), rope=rope)
        qa.qk_norm_rope(x, None, p, None, M, H, 0, D, norm=qa.NORM_NONE, rope=rope, cos=dev(np.cos(a).astype(np.float32)),
                        sin=dev(np.sin(a).astype(np.float32)))
        assert float((o.float() - p.float()).abs().max()) <= 2 * 2.0 ** -8 * float(x.abs().max()) * 2
