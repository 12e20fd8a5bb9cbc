"""A rotation that is asked for needs both of its tables."""
import ctypes

import pytest

import mixed_precision_quantized_act_amd as qa
from tests._call_cpu import calls
from tests.test_abi_attn_cpu import EINVAL, OK, P, _status

torch = pytest.importorskip("torch")

M, D = 3, 64


def _args(rope, cos, sin, pos=None):
    q, k, qo, ko = (torch.zeros((M, D), dtype=torch.bfloat16) for _ in range(4))
    return [q, k, qo, ko, M, 1, 1, D, 1, None, None, None, None, 1e-6, rope, cos, sin, pos, 0]


@pytest.mark.parametrize("rope", [qa.ROPE_PAIRS, qa.ROPE_HALVES])
def test_python_call(rope):
    c = calls()
    cos, sin = torch.ones((M, D // 2)), torch.zeros((M, D // 2))
    a = c.ok("qk_norm_rope", *_args(rope, cos, sin))
    assert (a[15], a[16], a[17]) == (cos.data_ptr(), sin.data_ptr(), M)
    c.refused("qk_norm_rope", *_args(rope, cos, None), match="cos")
    c.refused("qk_norm_rope", *_args(rope, None, sin), match="cos")
    c.refused("qk_norm_rope", *_args(rope, None, None), match="cos")
    # tables of no positions turn nothing, whether they have an address or not
    for e in (cos[:0], torch.zeros((0, D // 2))):
        for f in (sin[:0], torch.zeros((0, D // 2))):
            a = c.ok("qk_norm_rope", *_args(rope, e, f))
            assert (a[15], a[16], a[17]) == (None, None, 0)
    c.ok("qk_norm_rope", *_args(qa.ROPE_NONE, None, None))


def test_library():
    base = dict(q=P(0), ldq=256, Hq=4, k=P(1), ldk=128, Hk=2, M=0, D=64, norm=2, q_w=None, q_b=None, k_w=None,
                k_b=None, eps=1e-6, rope=1, cos=P(2), sin=P(3), P=0, pos=None, q_out=P(4), ldqo=256, k_out=P(5),
                ldko=128, stream=ctypes.c_void_p(None))
    for rope in (1, 2):
        for change, want in (({}, OK), ({"cos": None, "sin": None}, OK), ({"cos": None}, EINVAL), ({"sin": None}, EINVAL),
                             ({"cos": None, "P": 4}, EINVAL), ({"sin": None, "P": 4}, EINVAL),
                             ({"cos": None, "sin": None, "P": 4}, EINVAL)):
            assert _status("qk_norm_rope", {**base, "rope": rope, **change}) == want, change
