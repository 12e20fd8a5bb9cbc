"""qk_norm_rope refuses outputs that lie on what it reads beside the heads:
the norms' weights, the rotation's tables and the positions."""
import ctypes

import pytest

from tests.test_abi_attn_cpu import EALIAS, P, _status

M, D = 4, 64
OUT_BYTES = {"q_out": (M - 1) * 512 + 2 * 256, "k_out": (M - 1) * 256 + 2 * 128}
READ = {"q_w": 2 * D, "q_b": 2 * D, "k_w": 2 * D, "k_b": 2 * D, "cos": 10 * D // 2 * 4, "sin": 10 * D // 2 * 4, "pos": 4 * M}


@pytest.mark.parametrize("out", list(OUT_BYTES))
@pytest.mark.parametrize("read", list(READ))
def test_refused(out, read):
    base = dict(q=P(0), ldq=256, Hq=4, k=P(1), ldk=128, Hk=2, M=M, D=D, norm=2, q_w=P(6), q_b=P(7), k_w=P(8),
                k_b=P(9), eps=1e-6, rope=1, cos=P(2), sin=P(3), P=10, pos=P(10), q_out=P(4), ldqo=256, k_out=P(5),
                ldko=128, stream=None)
    at = base[out].value
    # the same place, what is read ending in the output's first bytes, and beginning in its last
    for place in (at, at - READ[read] + 16, at + OUT_BYTES[out] - 16):
        assert _status("qk_norm_rope", {**base, read: ctypes.c_void_p(place)}) == EALIAS, (out, read, hex(place))


@pytest.mark.parametrize("P_", [1 << 40, (1 << 63) - 1])
def test_long_tables(P_):
    """A table's length cannot wrap the check round."""
    base = dict(q=P(0), ldq=256, Hq=4, k=P(1), ldk=128, Hk=2, M=M, D=D, norm=0, q_w=None, q_b=None, k_w=None,
                k_b=None, eps=1e-6, rope=1, cos=P(3), sin=P(2), P=P_, pos=None, q_out=P(4), ldqo=256, k_out=P(5),
                ldko=128, stream=None)
    assert _status("qk_norm_rope", base) == EALIAS
