"""qlinear_w8a8 at sizes that take each of its ways (tests/_w8.py): sampled rows,
all columns, against the exact sums."""
import numpy as np
import pytest

from oracle import drafts as O
from oracle import gemm as G
from tests._attn import U_BF16, U_F32, bits, rng, val
from tests._gpu import dev, host, sample_rows, torch
from tests._w8 import PLANS

pytestmark = pytest.mark.gpu


def _rows(M, seed):
    """Rows at the edges of every kind of tile, and any."""
    edge = [r for t in (16, 32, 64, 128, 192, 256) for r in (t - 1, t, (M - 1) // t * t - 1, (M - 1) // t * t)]
    pick = set(sample_rows(M, 12, seed).tolist()) | {r for r in edge if 0 <= r < M}
    return np.array(sorted(pick))


@pytest.mark.parametrize("kind", list(PLANS))
@pytest.mark.parametrize("f32,gelu", [(True, False), (True, True), (False, False), (False, True)])
def test_plan(kind, f32, gelu):
    import mixed_precision_quantized_act_amd as qa
    t = torch()
    for M, N, K in PLANS[kind]:
        g = rng(431, M, N, K)
        a, w = (g.integers(-128, 128, s, dtype=np.int8) for s in ((M, K), (N, K)))
        a_s, w_s = ((2.0 ** g.uniform(-12, -2, n)).astype(np.float32) for n in (M, N))
        b = bits(g.standard_normal(N) * 50.0)
        ldy = N + 3
        y = t.full((M + 1, ldy), 7.0, dtype=t.float32 if f32 else t.bfloat16, device="cuda")
        ws = qa.qlinear_w8a8_workspace(M, N, K)
        args = dev(a), dev(a_s), dev(w), dev(w_s)
        kw = dict(bias=dev(b), out=qa.OUT_F32 if f32 else qa.OUT_BF16, epi=qa.EPI_GELU_TANH if gelu else qa.EPI_NONE)
        qa.qlinear_w8a8(*args, y, M, N, K, ws=t.full((ws,), 0xFF, dtype=t.uint8, device="cuda") if ws else None, **kw)
        # nothing beyond the output, and the same bits without a workspace
        assert bool((y[M] == 7.0).all()) and bool((y[:, N:] == 7.0).all())
        if ws:
            z = t.empty_like(y)
            qa.qlinear_w8a8(*args, z, M, N, K, **kw)
            assert t.equal(y[:M, :N], z[:M, :N])
        rows = _rows(M, N)
        got = y[dev(rows)]
        got = (host(got) if f32 else val(host(got))).astype(np.float64)[:, :N]
        v = O.int8_sums(a[rows], w) * a_s[rows].astype(np.float64)[:, None] * w_s.astype(np.float64)
        e = 3.001 * U_F32 * np.abs(v)
        v = v + val(b)
        e = e + 1.001 * U_F32 * (np.abs(v) + e)
        if gelu:
            e = 1.13 * e + 16 * U_F32 * np.abs(v)
            v = G.gelu_tanh(v)
        tol = e + (0 if f32 else U_BF16 * (np.abs(v) + e)) + 1e-37
        bad = ~(np.abs(got - v) <= tol)
        assert not bad.any(), ((M, N, K), np.argwhere(bad)[:4], got[bad][:4], v[bad][:4])
