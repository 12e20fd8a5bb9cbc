"""qlinear_w8a8's tiles one by one where every row is whole lines of 128 bytes, which go past the caches: every output,
against sums in float32 that are exact."""
import numpy as np
import pytest

from tests._attn import rng
from tests._gpu import dev, torch
from tests._w8 import PLANS

pytestmark = pytest.mark.gpu

SIZES = [s for kind, sizes in PLANS.items() if kind[0] == 0 and kind[3] == 0 for s in sizes]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_every_output(M, N, K, f32):
    import mixed_precision_quantized_act_amd as qa
    t = torch()
    g = rng(763, M, N, K)
    most = min(128, int((2 ** 24 / K) ** 0.5) - 1)
    assert K * most * most < 2 ** 24
    a, w = (g.integers(-most, most, s, dtype=np.int8) for s in ((M, K), (N, K)))
    a_s, w_s = ((2.0 ** g.uniform(-12, -2, n)).astype(np.float32) for n in (M, N))
    d, ldy, kind = [dev(x) for x in (a, a_s, w, w_s)], -(-N // 64) * 64, t.float32 if f32 else t.bfloat16
    y = t.full((M + 1, ldy), 7.0, dtype=kind, device="cuda")
    assert y.data_ptr() % 128 == 0 and ldy * y.element_size() % 128 == 0
    n = qa.qlinear_w8a8_workspace(M, N, K)
    qa.qlinear_w8a8(*d, y, M, N, K, out=qa.OUT_F32 if f32 else qa.OUT_BF16,
                    ws=t.empty(n, dtype=t.uint8, device="cuda") if n else None)
    assert bool((y[M] == 7.0).all()) and bool((y[:, N:] == 7.0).all())
    # (two products, each rounded to float32, and the output's rounding: the same steps)
    assert t.equal(y[:M, :N], (((d[0].float() @ d[2].float().t()) * d[3]) * d[1][:, None]).to(kind))
