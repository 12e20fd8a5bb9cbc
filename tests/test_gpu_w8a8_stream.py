"""qlinear_w8a8 where a workgroup of the stream has three tiles and more, whole lines past the caches among them:
every output, against sums in float32 that are exact (|sum| < 2^24)."""
import numpy as np
import pytest

from oracle import drafts as O
from tests._attn import U_BF16, U_F32, bits, rng
from tests._gpu import dev, torch
from tests._w8_stream import STREAMS

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("M,N,K,ldy,shape", STREAMS)
def test_every_output(M, N, K, ldy, shape, f32):
    import mixed_precision_quantized_act_amd as qa
    t = torch()
    assert K * 2 ** 14 < 2 ** 24
    g = rng(761, M, N, K)
    a, w = (g.integers(-128, 128, s, dtype=np.int8) for s in ((M, K), (N, K)))
    a_s, w_s = ((2.0 ** g.uniform(-12, -2, n)).astype(np.float32) for n in (M, N))
    d = [dev(x) for x in (a, a_s, w, w_s)]
    kind = t.float32 if f32 else t.bfloat16
    out = qa.OUT_F32 if f32 else qa.OUT_BF16
    y = t.full((M + 1, ldy), 7.0, dtype=kind, device="cuda")
    assert y.data_ptr() % 128 == 0
    qa.qlinear_w8a8(*d, y, M, N, K, out=out)
    assert bool((y[M] == 7.0).all()) and bool((y[:, N:] == 7.0).all())
    sums = d[0].float() @ d[2].float().t()
    for r in (0, M // 2, M - 1):
        assert np.array_equal(sums[r].cpu().numpy(), O.int8_sums(a[r:r + 1], w)[0])
    # (two products, each rounded to float32, and the output's rounding: the same steps)
    assert t.equal(y[:M, :N], ((sums * d[3]) * d[1][:, None]).to(kind))
    # the product with a_s and the bias: one more step in float32, of either sum
    b = dev(bits(g.standard_normal(N) * 50.0)).view(t.bfloat16)
    qa.qlinear_w8a8(*d, y, M, N, K, bias=b, out=out)
    v = (sums * d[3]).double() * d[1].double()[:, None]
    e = 1.001 * U_F32 * v.abs_()
    v = (sums * d[3]).double() * d[1].double()[:, None] + b.double()
    e += 1.001 * U_F32 * (v.abs() + e)
    if not f32:
        e += U_BF16 * (v.abs() + e)
    assert bool(((y[:M, :N].double() - v).abs() <= e).all())
    assert bool((y[M] == 7.0).all()) and bool((y[:, N:] == 7.0).all())


@pytest.mark.parametrize("M,N,K,ldy,shape", STREAMS[2:4])
def test_again_the_same_and_captured(M, N, K, ldy, shape):
    import mixed_precision_quantized_act_amd as qa
    t = torch()
    g = rng(762, M, N, K)
    d = [dev(g.integers(-128, 128, s, dtype=np.int8)) for s in ((M, K), (N, K))]
    s = [dev((2.0 ** g.uniform(-12, -2, n)).astype(np.float32)) for n in (M, N)]
    args, y = (d[0], s[0], d[1], s[1]), t.zeros((M, ldy), dtype=t.bfloat16, device="cuda")
    qa.qlinear_w8a8(*args, y, M, N, K)
    want = y.clone()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        qa.qlinear_w8a8(*args, y, M, N, K)
    for _ in range(4):
        y[:, :N] = 7.0
        graph.replay()
        t.cuda.synchronize()
        assert t.equal(y, want)
