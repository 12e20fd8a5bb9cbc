"""qlinear_bf16 at the weight sizes where a workgroup takes more weight rows,
and head norms of tiny heads."""
import numpy as np
import pytest

from oracle import attn as A
from tests._attn import U_BF16, U_F32, bits, rng, val
from tests._gpu import dev, host, torch
from tests.test_gpu_rows import _call, _case, _close, _expect

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [8191, 8192, 8209, 16383, 16384, 16391])
@pytest.mark.parametrize("M", [1, 2, 3, 5, 8, 9, 16, 17, 32])
def test_many_weight_rows(M, N):
    K = 272 if N % 2 else 256                 # a partial step of 256 elements, and none
    x, w, b = _case(M, N, K, 11)
    y, e = _expect(x, w, b, False)
    _close(_call(x, w, N, K, b, True), y, e, True)


@pytest.mark.parametrize("K", [16, 48, 240, 256, 2048, 2064, 4096, 4112, 6160])
@pytest.mark.parametrize("M", [1, 8, 9, 32])
def test_inner_sizes_around_the_waves_steps(M, K):
    x, w, b = _case(M, 50, K, 12)
    y, e = _expect(x, w, None, False)
    _close(_call(x, w, 50, K, None, False, ldx=K + 24), y, e, False)


@pytest.mark.parametrize("M", [1, 4, 16, 32])
def test_a_row_that_is_not_finite_stays_alone(M):
    x, w, _ = _case(M, 8200, 528, 13)
    good = _call(x, w, 8200, 528, None, True)
    x[M - 1, 5] = 0x7FC0                      # NaN
    got = _call(x, w, 8200, 528, None, True)
    assert np.isnan(got[M - 1]).all()
    assert np.array_equal(got[:M - 1], good[:M - 1])


@pytest.mark.parametrize("exponent", [-40, -60])
@pytest.mark.parametrize("norm", [1, 2])
def test_norm_of_tiny_heads_without_eps(exponent, norm):
    """Variances down to 2^-120, where an inverse root of a float32 needs scaling."""
    import mixed_precision_quantized_act_amd as qa
    t = torch()
    M, H, D = 5, 3, 64
    g = rng(503, exponent + 100, norm)
    x = bits(g.standard_normal((M, H * D)) * 2.0 ** exponent)
    o = t.empty((M, H * D), dtype=t.bfloat16, device="cuda")
    qa.qk_norm_rope(dev(x).view(t.bfloat16), None, o, None, M, H, 0, D, norm=norm, eps=0.0)
    xv = val(x).reshape(M, H, D)
    y = A.norm_rope(xv, norm, None, None, 0.0, 0, None, None, None)
    # the output's rounding, and D + 16 half steps of sums and products of
    # values of at most sqrt(D) deviations
    tol = U_BF16 * np.abs(y) + 4 * (D + 16) * U_F32 * np.sqrt(D)
    assert np.all(np.abs(val(host(o)).reshape(M, H, D) - y) <= tol)


@pytest.mark.parametrize("N", [1, 510, 1024, 1030, 2050, 2064, 4096, 4100])
@pytest.mark.parametrize("M", [8, 9, 15, 16, 17, 24, 25, 31, 32])
def test_rows_shared_out_over_workgroups(M, N):
    """8, 16 or 32 rows to a workgroup, by the weight's size; bf16 rows of a wider output."""
    x, w, b = _case(M, N, 288, 14)
    y, e = _expect(x, w, b, False)
    _close(_call(x, w, N, 288, b, False, ldx=296, ldy=N + 3), y, e, False)


@pytest.mark.parametrize("N", [8200, 12290])
def test_large_weights(N):
    """Sizes at which a workgroup takes 32 and 64 weight rows, of one weight for all row counts."""
    K = 2064
    x, w, b = _case(32, N, K, 15)
    y, e = _expect(x, w, b, True)
    for M in (1, 3, 8, 9, 16, 17, 32):
        _close(_call(x[:M], w, N, K, b, True, gelu=True), y[:M], e[:M], True)
