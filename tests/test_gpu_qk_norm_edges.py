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


SPECIAL = np.array([0x7F80, 0xFF80, 0x7F7F, 0xFF7F, 0x8000, 0x0000, 0x0001, 0x8001, 0x0080, 0x3F80], np.uint16)


@pytest.mark.parametrize("D", [16, 64, 80, 128, 256])
@pytest.mark.parametrize("rope", [1, 2])
def test_tokens_that_are_not_turned_are_passed_on(rope, D):
    """Without a norm every element keeps its bits: infinities beside finite
    elements, signed zeros, the smallest and largest values.  Tokens that are
    turned stand between them."""
    qa, t = _qa(), torch()
    M, H = 7, 3
    g = rng(505, rope, D)
    x = bits(g.standard_normal((M, H * D)))
    x[::2] = np.where(g.random((4, H * D)) < 0.5, SPECIAL[g.integers(0, len(SPECIAL), (4, H * D))], x[::2])
    pos = np.array([-1, 0, 2 ** 31 - 1, 3, 4, 2, -2 ** 31], np.int32)
    cos, sin = _tables(4, D, 3)
    o = t.empty((M, H * D), dtype=t.bfloat16, device="cuda")
    k = t.empty_like(o)
    xd = dev(x).view(t.bfloat16)
    qa.qk_norm_rope(xd, xd.clone(), o, k, M, H, H, D, norm=qa.NORM_NONE, rope=rope, cos=dev(cos), sin=dev(sin),
                    pos=dev(pos))
    t.cuda.synchronize()
    for out in (host(o), host(k)):
        assert np.array_equal(out[::2], x[::2])
        xv = val(x[1::2]).reshape(3, H, D)
        y = A.norm_rope(xv, 0, None, None, 0.0, rope, cos, sin, pos[1::2])
        # two products of half a step each and one of their sum, on a value of at most twice the largest
        tol = U_BF16 * np.abs(y) + 4 * 2.0 ** -24 * np.abs(xv).max()
        assert np.all(np.abs(val(out[1::2]).reshape(3, H, D) - y) <= tol)


@pytest.mark.parametrize("rope", [1, 2])
def test_an_infinite_weight_reaches_its_own_element_only(rope):
    """A normed head of a token that is not turned: one element infinite, its partner as it was."""
    qa, t = _qa(), torch()
    D = 64
    g = t.Generator(device="cuda").manual_seed(4)
    x = t.randn((2, 2 * D), generator=g, device="cuda").bfloat16()
    w = t.ones(D, dtype=t.bfloat16, device="cuda")
    kw = dict(norm=qa.NORM_RMS, rope=rope, cos=t.ones((2, D // 2), device="cuda"), sin=t.ones((2, D // 2), device="cuda"),
              pos=t.full((2,), -1, dtype=t.int32, device="cuda"))
    a, b = t.empty_like(x), t.empty_like(x)
    qa.qk_norm_rope(x, None, a, None, 2, 2, 0, D, q_w=w, **kw)
    w[10] = float("inf")
    qa.qk_norm_rope(x, None, b, None, 2, 2, 0, D, q_w=w, **kw)
    same = (a == b).view(2, 2, D)
    assert not same[..., 10].any() and same[..., [i for i in range(D) if i != 10]].all()
    assert b.view(2, 2, D)[..., 10].isinf().all()
