"""qk_norm_rope: what may lie beside its outputs, and tokens that are not turned."""
import numpy as np
import pytest

from oracle import attn as A
from tests._attn import U_BF16, bits, rng, val
from tests._gpu import dev, host, torch
from tests.test_gpu_qk_norm import _tables, _tol

pytestmark = pytest.mark.gpu


def _qa():
    import mixed_precision_quantized_act_amd as qa
    return qa


def test_weights_in_a_row_of_the_outputs_buffer():
    """What is read may share the output's buffer at columns that are not written."""
    qa, t = _qa(), torch()
    M, H, D = 5, 2, 64
    g = rng(504)
    x = bits(g.standard_normal((M, H * D)))
    w, b = bits(1 + 0.2 * g.standard_normal(D)), bits(0.1 * g.standard_normal(D))
    o = t.full((M, H * D + 2 * D), 7.0, dtype=t.bfloat16, device="cuda")
    o[2, H * D:H * D + D] = dev(w).view(t.bfloat16)
    o[4, H * D + D:] = dev(b).view(t.bfloat16)
    before = o.clone()
    qa.qk_norm_rope(dev(x).view(t.bfloat16), None, o, None, M, H, 0, D, norm=qa.NORM_LAYER,
                    q_w=o[2, H * D:H * D + D], q_b=o[4, H * D + D:], eps=1e-5)
    t.cuda.synchronize()
    xv = val(x).reshape(M, H, D)
    y = A.norm_rope(xv, 2, val(w), val(b), 1e-5, 0, None, None, None)
    got = val(host(o[:, :H * D])).reshape(M, H, D)
    assert np.all(np.abs(got - y) <= _tol(y, xv, val(w), val(b), 1e-5, D))
    assert t.equal(o[:, H * D:], before[:, H * D:])
