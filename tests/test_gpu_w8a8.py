"""qlinear_w8a8 (INT8 activations against an INT8 weight) against the exact
sums of its codes, element by element."""
import numpy as np
import pytest

from oracle import drafts as O
from oracle import gemm as G
from tests._attn import U_BF16, U_F32, bits, rng, val
from tests._gpu import dev, host, torch

pytestmark = pytest.mark.gpu


def _qa():
    import mixed_precision_quantized_act_amd as qa
    return qa


def _case(M, N, K, seed=0, extreme=False):
    g = rng(411, M, N, K, seed)
    draw = (lambda s: g.choice(np.array([-128, 127], np.int8), s)) if extreme else \
        (lambda s: g.integers(-128, 128, s, dtype=np.int8))
    scales = lambda n: (2.0 ** g.uniform(-12, 2, n)).astype(np.float32)  # noqa: E731
    return draw((M, K)), scales(M), draw((N, K)), scales(N), bits(g.standard_normal(N) * 50.0)


def _expect(c, bias, gelu):
    """(y, bound on the float32 error) in float64: the sum rounded to float32,
    two products, the bias, one rounding each; GELU has slope below 1.13 and
    adds at most 8 steps of its argument."""
    a, a_s, w, w_s, b = c
    y = O.int8_sums(a, w) * a_s.astype(np.float64)[:, None] * w_s.astype(np.float64)
    e = 3.001 * U_F32 * np.abs(y)
    if bias:
        y = y + val(b)
        e = e + 1.001 * U_F32 * (np.abs(y) + e)
    if gelu:
        e = 1.13 * e + 16 * U_F32 * np.abs(y)
        y = G.gelu_tanh(y)
    return y, e


def _device(c):
    a, a_s, w, w_s, b = c
    return [dev(a), dev(a_s), dev(w), dev(w_s), dev(b)]


def _call(c, bias=False, f32=False, gelu=False, ldy=None, ws="full", y_off=0, stream=None):
    qa, t = _qa(), torch()
    (M, K), N = c[0].shape, c[2].shape[0]
    ldy = ldy or N
    y = t.full(((M + 1) * ldy + y_off,), 7.0, dtype=t.float32 if f32 else t.bfloat16, device="cuda")
    y = y[y_off:].view(M + 1, ldy)
    n = qa.qlinear_w8a8_workspace(M, N, K) if ws == "full" else ws
    d = _device(c)
    qa.qlinear_w8a8(*d[:4], y, M, N, K, bias=d[4] if bias else None, out=qa.OUT_F32 if f32 else qa.OUT_BF16,
                    epi=qa.EPI_GELU_TANH if gelu else qa.EPI_NONE, ldy=ldy,
                    ws=t.full((n,), 0xFF, dtype=t.uint8, device="cuda") if n else None, stream=stream)
    t.cuda.synchronize()
    yh = host(y) if f32 else val(host(y))
    assert np.all(yh[M] == 7.0) and np.all(yh[:M, N:] == 7.0)      # nothing beyond the output
    return yh[:M, :N].astype(np.float64)


def _check(c, bias=False, f32=False, gelu=False, **kw):
    got = _call(c, bias, f32, gelu, **kw)
    y, e = _expect(c, bias, gelu)
    tol = e + (0 if f32 else U_BF16 * (np.abs(y) + e)) + 1e-37
    bad = ~(np.abs(got - y) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], y[bad][:4], tol[bad][:4])
    return got


SIZES = [(1, 1, 16), (1, 16, 16), (2, 17, 32), (3, 15, 48), (1, 33, 112), (7, 130, 64), (16, 64, 128), (17, 129, 144),
         (31, 300, 80), (32, 128, 256), (33, 127, 272), (48, 1000, 528), (64, 256, 1024), (65, 255, 1040), (100, 100, 16),
         (127, 385, 320), (128, 128, 64), (129, 257, 208), (255, 511, 96), (256, 256, 512), (257, 513, 176),
         (300, 70, 2048), (520, 640, 336), (1000, 33, 400)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_sizes(M, N, K):
    c = _case(M, N, K)
    _check(c, f32=True)
    _check(c, bias=True, ldy=N + 5)
    _check(c, gelu=True, bias=True, ldy=(N + 15) // 8 * 8)


@pytest.mark.parametrize("M,N,K", [(1, 64, 8192), (40, 70, 4112), (300, 200, 4096), (64, 1920, 7680)])
@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("gelu", [True, False])
def test_long_sums_and_epilogues(M, N, K, f32, bias, gelu):
    _check(_case(M, N, K), bias, f32, gelu)


@pytest.mark.parametrize("M", [1, 33, 130])
def test_largest_sums(M):
    """All codes -128 or 127 over the longest K: sums up to 2^31 - 2^18."""
    K = (1 << 17) - 16
    c = _case(M, 40, K, extreme=True)
    _check(c, f32=True)
    a, w = np.full((M, K), -128, np.int8), np.full((40, K), -128, np.int8)
    got = _call((a, np.ones(M, np.float32), w, np.ones(40, np.float32), c[4]), f32=True)
    assert np.all(got == 16384.0 * K)                   # (17 significant bits: exact in float32)


def test_exact_in_float32():
    """Sums below 2^24 and scales that are powers of two: every bit."""
    for M, N, K in ((5, 40, 1024), (70, 300, 512), (260, 270, 256)):
        a, a_s, w, w_s, b = _case(M, N, K)
        a_s, w_s = 2.0 ** np.floor(np.log2(a_s)), 2.0 ** np.floor(np.log2(w_s))
        c = (a, a_s.astype(np.float32), w, w_s.astype(np.float32), b)
        assert np.array_equal(_call(c, f32=True), _expect(c, False, False)[0])


@pytest.mark.parametrize("M,N,K", [(1, 300, 2048), (64, 500, 4096), (200, 129, 6000), (513, 600, 2048)])
def test_any_workspace_gives_the_same_bits(M, N, K):
    c = _case(M, N, K)
    full = _call(c, bias=True, f32=True)
    n = _qa().qlinear_w8a8_workspace(M, N, K)
    for ws in {0, 16, n // 2 // 16 * 16, n + 4096}:
        assert np.array_equal(_call(c, bias=True, f32=True, ws=ws), full)
    assert np.array_equal(_call(c, bias=True, f32=True), full)


@pytest.mark.parametrize("y_off,ldy", [(1, 130), (2, 131), (4, 132), (8, 136), (8, 129)])
def test_outputs_of_any_alignment(y_off, ldy):
    for M in (3, 70):
        c = _case(M, 129, 160)
        _check(c, bias=True, y_off=y_off, ldy=ldy)
        _check(c, f32=True, y_off=y_off, ldy=ldy)


def test_scales_that_are_zero_or_not_finite():
    """A row or column of scale zero gives zeros, one that is no number gives NaN; the others keep theirs."""
    for M in (5, 90):
        c = list(_case(M, 70, 96))
        c[1], c[3] = c[1].copy(), c[3].copy()
        c[1][1], c[1][2], c[3][4], c[3][5] = 0.0, np.nan, 0.0, np.inf
        got = _call(c, f32=True)
        want = _call(_case(M, 70, 96), f32=True)
        rows, cols = [i for i in range(M) if i not in (1, 2)], [j for j in range(70) if j not in (4, 5)]
        assert np.array_equal(got[np.ix_(rows, cols)], want[np.ix_(rows, cols)])
        assert np.all(got[1, cols] == 0) and np.all(np.isnan(got[2])) and np.all(got[rows, 4] == 0)
        assert np.all(np.isinf(got[rows, 5]) | np.isnan(got[rows, 5]))


def test_against_act_quant():
    """Codes and scales as act_quant makes them, both sides: the library's chain
    against the float64 product of what they stand for."""
    qa, t = _qa(), torch()
    M, N, K = 70, 200, 320
    g = rng(412)
    out = []
    for rows, gain in ((M, 3.0), (N, 0.02)):
        x = dev(bits(g.standard_normal((rows, K)) * gain)).view(t.bfloat16)
        q, s = qa.empty_int8_act(rows, K)
        qa.act_quant(qa.INT8, x, q, s)
        out += [host(q, np.int8), host(s)]
    _check((*out, bits(g.standard_normal(N))), bias=True, gelu=True)


def test_no_rows_no_columns_and_gate():
    qa, t = _qa(), torch()
    for M, N in ((0, 32), (3, 0), (0, 0)):
        y = t.full((4, 40), 7.0, dtype=t.bfloat16, device="cuda")
        qa.qlinear_w8a8(t.zeros((M, 64), dtype=t.int8, device="cuda"), t.ones(M, device="cuda"),
                        t.zeros((N, 64), dtype=t.int8, device="cuda"), t.ones(N, device="cuda"), y, M, N, 64)
        assert (y == 7.0).all()
    for M in (3, 64, 300):
        c = _device(_case(M, 200, 2048))
        y = t.full((M, 200), 7.0, dtype=t.bfloat16, device="cuda")
        ws = t.empty(max(16, qa.qlinear_w8a8_workspace(M, 200, 2048)), dtype=t.uint8, device="cuda")
        with qa.gate(t.zeros(1, dtype=t.uint8, device="cuda"), 1):
            qa.qlinear_w8a8(*c[:4], y, M, 200, 2048, ws=ws)
        assert (y == 7.0).all()


@pytest.mark.parametrize("M", [1, 64, 300])
def test_streams_and_graphs(M):
    """The same bits on a second stream and from a graph that is replayed with
    other inputs, eager calls (a workspace of their own) between."""
    qa, t = _qa(), torch()
    N, K = 500, 4096
    sets = [_device(_case(M, N, K, s)) for s in range(3)]
    n = max(16, qa.qlinear_w8a8_workspace(M, N, K))
    ws = [t.full((n,), 0xFF, dtype=t.uint8, device="cuda") for _ in range(2)]
    y = [t.empty((M, N), dtype=t.bfloat16, device="cuda") for _ in range(2)]
    want = []
    for s in sets:
        qa.qlinear_w8a8(*s[:4], y[0], M, N, K, bias=s[4], ws=ws[0])
        want.append(y[0].clone())
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        y[0].zero_()
        qa.qlinear_w8a8(*sets[1][:4], y[0], M, N, K, bias=sets[1][4], ws=ws[0])
    t.cuda.synchronize()
    assert t.equal(y[0], want[1])
    held = [x.clone() for x in sets[0]]
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        qa.qlinear_w8a8(*held[:4], y[0], M, N, K, bias=held[4], ws=ws[0])
    for i in (0, 1, 2, 1, 0):
        for h, s in zip(held, sets[i]):
            h.copy_(s)
        graph.replay()
        j = (i + 1) % 3
        qa.qlinear_w8a8(*sets[j][:4], y[1], M, N, K, bias=sets[j][4], ws=ws[1])
        assert t.equal(y[0], want[i]) and t.equal(y[1], want[j])
