"""qlinear_bf16 (a few bf16 rows against an NVFP4 weight) against the
float64 product of the same values, element by element."""
import numpy as np
import pytest

from oracle import attn as A
from oracle import formats as F
from oracle import gemm as G
from oracle import quant as Q
from tests._attn import U_BF16, U_F32, bits, rng, val
from tests._gpu import dev, host, torch

pytestmark = pytest.mark.gpu


def _qa():
    import mixed_precision_quantized_act_amd as qa
    return qa


def _case(M, N, K, seed=0, outliers=True):
    g = rng(401, M, N, K, seed)
    x = g.standard_normal((M, K))
    if outliers:
        x[:, g.integers(0, K, max(1, K // 100))] *= 30.0
    w = Q.nvfp4_encode(bits(g.standard_normal((N, K)) * 0.02))
    return bits(x), w, bits(g.standard_normal(N) * 0.1)


def _expect(x, w, bias, gelu):
    """(y, bound on the float32 error) in float64.  Each output is K exact
    products summed in float32 in some order: at most K half steps of the
    sum of their absolute values (a whole step each where the adder
    truncates), the group scale's multiply-adds, then one rounding each by
    the tensor scale and the bias; GELU has slope below 1.13 and adds at most
    8 steps of its argument."""
    wv = A.unscaled(w[0], w[1]) * float(w[2])
    xv = val(x)
    y = xv @ wv.T
    K = xv.shape[1]
    e = 2 * U_F32 * (K + K / 16 + 8) * (np.abs(xv) @ np.abs(wv).T)
    if bias is not None:
        y = y + val(bias)[None]
        e = e + U_F32 * np.abs(y)
    if gelu:
        e = 1.13 * e + 16 * U_F32 * np.abs(y)
        y = G.gelu_tanh(y)
    return y, e


def _call(x, w, N, K, bias=None, f32=False, gelu=False, ldx=None, ldy=None, ws_off=0, stream=None):
    qa, t = _qa(), torch()
    M = x.shape[0]
    ldx, ldy = ldx or K, ldy or N
    xd = t.full((M, ldx), float("nan"), dtype=t.bfloat16, device="cuda")
    xd[:, :K] = dev(x).view(t.bfloat16)
    y = t.full((M + 1, ldy), 7.0, dtype=t.float32 if f32 else t.bfloat16, device="cuda")
    s = t.empty(w[1].size + ws_off, dtype=t.uint8, device="cuda")[ws_off:]
    s.copy_(dev(w[1]).reshape(-1))
    qa.qlinear_bf16(xd, dev(w[0]), s, dev(np.array([w[2]], np.float32)), y, M, N, K,
                    bias=None if bias is None else dev(bias), out=qa.OUT_F32 if f32 else qa.OUT_BF16,
                    epi=qa.EPI_GELU_TANH if gelu else qa.EPI_NONE, ldy=ldy, stream=stream)
    t.cuda.synchronize()
    yh = host(y) if f32 else val(host(y))
    assert np.all(yh[M] == 7.0) and np.all(yh[:M, N:] == 7.0)      # nothing beyond the output
    return yh[:M, :N].astype(np.float64)


def _close(got, y, e, f32):
    tol = e + (0 if f32 else U_BF16 * (np.abs(y) + e)) + 1e-37
    bad = np.abs(got - y) > tol
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], y[bad][:4], tol[bad][:4])


@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 16, 16), (2, 17, 32), (3, 15, 48), (1, 33, 112),
                                   (8, 64, 128), (9, 40, 144), (16, 31, 240), (17, 48, 256), (32, 130, 272),
                                   (24, 16, 1920), (5, 257, 1024), (1, 100, 4112), (32, 5, 2064), (12, 96, 1040)])
@pytest.mark.parametrize("f32", [True, False])
def test_rows_against_float64(M, N, K, f32):
    x, w, b = _case(M, N, K)
    _close(_call(x, w, N, K, f32=f32), *_expect(x, w, None, False), f32)


@pytest.mark.parametrize("gelu", [False, True])
@pytest.mark.parametrize("M,N,K", [(2, 1152, 512), (7, 65, 1936), (32, 33, 528)])
def test_rows_bias_gelu_strides(M, N, K, gelu):
    x, w, b = _case(M, N, K, 1)
    y, e = _expect(x, w, b, gelu)
    for f32 in (True, False):
        _close(_call(x, w, N, K, b, f32, gelu, ldx=K + 24, ldy=N + 3, ws_off=1), y, e, f32)


def test_rows_real_sizes():
    for M, N, K in ((2, 11520, 512), (16, 1920, 7680), (1, 7680, 1920)):
        x, w, b = _case(M, N, K, 2)
        _close(_call(x, w, N, K, b, True), *_expect(x, w, b, False), True)


def test_rows_values_at_the_edges():
    """Large and tiny activations in one row, group scales of every code, zero groups, a zero weight."""
    M, N, K = 3, 127, 2032
    g = rng(77)
    x = bits(g.standard_normal((M, K)) * 2.0 ** g.integers(-60, 60, (M, K)))
    codes = g.integers(0, 256, (N, K // 2), dtype=np.uint8)
    scales = (np.arange(N * (K // 16)) % 0x7F).astype(np.uint8).reshape(N, K // 16)
    scales[5] = 0
    w = (codes, scales, np.float32(2.0 ** -7))
    _close(_call(x, w, N, K, f32=True), *_expect(x, w, None, False), True)
    w0 = (np.zeros_like(codes), np.zeros_like(scales), np.float32(0.0))
    assert np.all(_call(x, w0, N, K, f32=True) == 0.0)


def test_rows_not_finite():
    """An infinity reaches the outputs of its own row alone, as in a plain product."""
    M, N, K = 4, 40, 256
    x, w, _ = _case(M, N, K, 3)
    x[2, 100] = 0x7F80                                     # +inf
    wv = A.unscaled(w[0], w[1]) * float(w[2])
    with np.errstate(invalid="ignore"):
        y = val(x) @ wv.T
    got = _call(x, w, N, K, f32=True)
    assert np.array_equal(np.isnan(got[2]), wv[:, 100] == 0)
    assert np.array_equal(got[2][wv[:, 100] != 0], y[2][wv[:, 100] != 0])
    xs, e = _expect(x[[0, 1, 3]], w, None, False)
    _close(got[[0, 1, 3]], xs, e, True)


def test_rows_repeat_gate_stream():
    """The same bits on every call and on another stream; a closed gate leaves the output."""
    qa, t = _qa(), torch()
    M, N, K = 6, 200, 1040
    x, w, b = _case(M, N, K, 4)
    first = _call(x, w, N, K, b, True)
    st = t.cuda.Stream()
    st.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(st):
        assert np.array_equal(first, _call(x, w, N, K, b, True))
    gate = t.tensor([2], dtype=t.uint8, device="cuda")
    with qa.gate(gate, 1):
        assert np.all(_call(x, w, N, K, b, True) == 7.0)
    with qa.gate(gate, 2):
        assert np.array_equal(first, _call(x, w, N, K, b, True))


def test_rows_nothing_to_do():
    qa, t = _qa(), torch()
    x, w, b = _case(1, 16, 64, 5)
    y = t.full((4, 16), 7.0, dtype=t.float32, device="cuda")
    a = (dev(x).view(t.bfloat16), dev(w[0]), dev(w[1]), dev(np.array([w[2]], np.float32)), y)
    qa.qlinear_bf16(*a, 0, 16, 64, out=qa.OUT_F32)
    qa.qlinear_bf16(*a, 1, 0, 64, out=qa.OUT_F32)
    t.cuda.synchronize()
    assert (y == 7.0).all()
