"""rope_freqs from Python: sizes and kinds that do not fit 32 bits are refused, not cut to their lowest ones."""
import pytest

import mixed_precision_quantized_act_amd as qa
from tests.test_abi_attn_cpu import EINVAL, ESHAPE


@pytest.mark.parametrize("R", [2 ** 32 + 16, -2 ** 32 + 16, 2 ** 64 + 32, -2 ** 64 + 2, 2 ** 31, -2, 0, 1, 65537, 65538])
def test_sizes(R):
    with pytest.raises(qa.QactError) as e:
        qa.rope_freqs(R)
    assert e.value.status == ESHAPE


@pytest.mark.parametrize("stretch", [-1, 4, 2 ** 32, 2 ** 32 + 1, -2 ** 32, 2 ** 64 + 3])
def test_kinds(stretch):
    with pytest.raises(qa.QactError) as e:
        qa.rope_freqs(64, stretch=stretch)
    assert e.value.status == EINVAL


def test_the_largest_and_the_smallest():
    assert qa.rope_freqs(65536)[0].shape == (32768,) and qa.rope_freqs(2)[0].shape == (1,)


@pytest.mark.parametrize("R,factor", [(4, 1e155), (64, 1e300), (6, 1e204)])
def test_a_stretched_base_beyond_float64(R, factor):
    """(Its frequencies would be zeros but for the first.)"""
    with pytest.raises(qa.QactError) as e:
        qa.rope_freqs(R, 10000.0, qa.STRETCH_BASE, factor=factor)
    assert e.value.status == EINVAL
    f, _ = qa.rope_freqs(R, 10000.0, qa.STRETCH_BASE, factor=1e100)
    assert (f > 0).all()
