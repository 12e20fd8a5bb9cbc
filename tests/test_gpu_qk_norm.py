"""qk_norm_rope against its float64 definition."""
import numpy as np
import pytest

from oracle import attn as A
from tests._attn import U_BF16, U_F32, bits, rng, val
from tests._gpu import dev, host, torch

pytestmark = pytest.mark.gpu


def _qa():
    import mixed_precision_quantized_act_amd as qa
    return qa


def _tables(P, D, first=0):
    a = (first + np.arange(P))[:, None] * 10000.0 ** (-np.arange(D // 2) / (D // 2))
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def _tol(y, x, w, b, eps, D):
    """Rounding of the output; float32 before it: sums of D terms, 8 more
    operations, on a value of at most (max |x| / deviation) |w| + |b|; the
    rotation adds two such terms."""
    sd = np.sqrt(x.var(-1, keepdims=True) + eps)
    rms = np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    size = 2 * np.abs(x).max(-1, keepdims=True) / np.minimum(sd, rms) * np.abs(w).max() + np.abs(b).max()
    f = (2 * D + 32) * 2 * U_F32 * size
    return U_BF16 * np.abs(y) + 2 * f


def _run(M, Hq, Hk, D, norm, rope, pos=None, P=None, weights=True, bias=True, in_place=False, pad=0, seed=0,
         offset=0.0):
    qa, t = _qa(), torch()
    g = rng(501, M, Hq, Hk, D, norm, rope, seed)
    width = (Hq + 2 * Hk) * D + pad
    qkv = bits(g.standard_normal((M, width)) * 2.0 + offset)
    ws = [bits(1 + 0.2 * g.standard_normal(D)) if weights and norm else None for _ in range(2)]
    bs = [bits(0.1 * g.standard_normal(D)) if bias and norm else None for _ in range(2)]
    P = M if P is None else P
    cos, sin = _tables(P, D, 5)
    d = dev(qkv).view(t.bfloat16)
    nq, nk = Hq * D, Hk * D
    q, k = d[:, :nq], d[:, nq:nq + nk]
    if in_place:
        qo, ko = q, k
    else:
        qo = t.full((M + 1, nq + 8), 7.0, dtype=t.bfloat16, device="cuda")
        ko = t.full((M + 1, nk + 16), 7.0, dtype=t.bfloat16, device="cuda")
    tens = lambda a: None if a is None else dev(a)  # noqa: E731
    kw = dict(cos=dev(cos), sin=dev(sin), pos=tens(None if pos is None else np.asarray(pos, np.int32))) if rope else {}
    qa.qk_norm_rope(q if Hq else None, k if Hk else None, qo if Hq else None, ko if Hk else None, M, Hq, Hk, D,
                    norm=norm, q_w=tens(ws[0]) if Hq else None, q_b=tens(bs[0]) if Hq else None,
                    k_w=tens(ws[1]) if Hk else None, k_b=tens(bs[1]) if Hk else None, eps=1e-5, rope=rope, **kw)
    t.cuda.synchronize()
    at = np.arange(M) if pos is None else np.asarray(pos)
    for i, (H, o, lo) in enumerate(((Hq, qo, 0), (Hk, ko, nq))):
        if not H:
            continue
        x = val(qkv[:, lo:lo + H * D]).reshape(M, H, D)
        w = val(ws[i]) if ws[i] is not None else np.ones(D)
        b = val(bs[i]) if bs[i] is not None else np.zeros(D)
        y = A.norm_rope(x, norm, w, b, 1e-5, rope, cos, sin, at)
        oh = val(host(o))
        got = oh[:M, :H * D].reshape(M, H, D)
        tol = _tol(y, x, w, b, 1e-5, D) if norm else U_BF16 * np.abs(y) + 4 * U_F32 * np.abs(x).max()
        bad = np.abs(got - y) > tol
        assert not bad.any(), (i, np.argwhere(bad)[:4], got[bad][:4], y[bad][:4], tol[bad][:4])
        if not in_place:
            assert np.all(oh[M] == 7.0) and np.all(oh[:, H * D:] == 7.0)
    if in_place:        # the values in the same rows stay
        assert np.array_equal(host(d)[:, nq + nk:], qkv[:, nq + nk:])


@pytest.mark.parametrize("D", [16, 32, 48, 64, 80, 96, 112, 128, 144, 192, 256])
@pytest.mark.parametrize("norm,rope", [(2, 1), (1, 2), (2, 2), (1, 1), (0, 1), (0, 2), (2, 0), (1, 0)])
def test_head_sizes(D, norm, rope):
    _run(13, 5, 3, D, norm, rope)


@pytest.mark.parametrize("M,Hq,Hk", [(1, 1, 0), (1, 0, 1), (1, 30, 30), (2, 7, 1), (9, 32, 8), (67, 24, 24),
                                     (300, 30, 30), (3, 129, 2)])
def test_heads_and_tokens(M, Hq, Hk):
    _run(M, Hq, Hk, 64, 2, 1)
    _run(M, Hq, Hk, 128, 1, 2, weights=M > 2, bias=False)


@pytest.mark.parametrize("rope", [1, 2])
def test_positions(rope):
    # text tokens first (-1), repeated and descending positions, some past the table
    pos = [-1, -1, -5, 0, 3, 3, 2, 1, 0, 11, 12, 13, 2 ** 31 - 1, -2 ** 31]
    _run(len(pos), 3, 2, 64, 2, rope, pos=pos, P=12)
    _run(4, 3, 2, 64, 2, rope, pos=[0, 1, 2, 3], P=0)


@pytest.mark.parametrize("rope", [0, 1, 2])
def test_in_place_within_one_projection(rope):
    _run(37, 6, 2, 64, 2, rope, in_place=True, pad=8)


def test_constant_and_zero_heads():
    """A head of equal values has no deviation: the bias alone, through eps."""
    qa, t = _qa(), torch()
    x = t.zeros((3, 128), dtype=t.bfloat16, device="cuda")
    x[1] = 2.0
    b = t.arange(64, device="cuda").bfloat16()
    o = t.empty_like(x)
    qa.qk_norm_rope(x, None, o, None, 3, 2, 0, 64, norm=qa.NORM_LAYER, q_b=b, eps=1e-6)
    assert (o.view(3, 2, 64) == b).all()


def test_not_finite_stays_in_its_head():
    qa, t = _qa(), torch()
    g = t.Generator(device="cuda").manual_seed(3)
    x = t.randn((5, 4 * 64), generator=g, device="cuda").bfloat16()
    y = t.empty_like(x)
    qa.qk_norm_rope(x, None, y, None, 5, 4, 0, 64, norm=qa.NORM_RMS)
    x2, y2 = x.clone(), t.empty_like(x)
    x2[2, 70] = float("inf")
    x2[3, 10] = float("nan")
    qa.qk_norm_rope(x2, None, y2, None, 5, 4, 0, 64, norm=qa.NORM_RMS)
    same = (y == y2).view(5, 4, 64).all(-1)
    want = t.ones((5, 4), dtype=t.bool, device="cuda")
    want[2, 1] = want[3, 0] = False
    assert (same == want).all() and y2[3, :64].isnan().all()


def test_gate():
    qa, t = _qa(), torch()
    x = t.randn((4, 64), device="cuda").bfloat16()
    y = t.full_like(x, 7.0)
    with qa.gate(t.zeros(1, dtype=t.uint8, device="cuda"), 1):
        qa.qk_norm_rope(x, None, y, None, 4, 1, 0, 64)
    assert (y == 7.0).all()
