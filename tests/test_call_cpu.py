"""The compiled calls without a GPU: they load, count their arguments and end
in a Python error, not in a crash."""
import pytest

import mixed_precision_quantized_act_amd as qa


def test_calls_end_in_errors():
    torch = pytest.importorskip("torch")
    from mixed_precision_quantized_act_amd import _lib
    m = _lib._native()
    for name, n in (("qlinear_bf16", 14), ("qk_norm_rope", 19), ("kv4_append", 14), ("kv4_read", 14),
                    ("attn_kv4", 18), ("attn_cross", 15)):
        with pytest.raises(TypeError):
            getattr(m, name)()
        with pytest.raises(TypeError):
            getattr(m, name)(*[None] * (n + 1))
        with pytest.raises((ValueError, RuntimeError, TypeError)):
            getattr(m, name)(*[None] * n)
        with pytest.raises((ValueError, RuntimeError, TypeError)):
            getattr(m, name)(*["no tensor"] * (n - 1), 0)
    x = torch.zeros((1, 64), dtype=torch.bfloat16)
    w = torch.zeros((32, 32), dtype=torch.uint8)
    with pytest.raises((ValueError, RuntimeError)):
        qa.qlinear_bf16(x, w, w, torch.ones(1), x, 1, 32, 64)
    with pytest.raises((ValueError, RuntimeError)):
        qa.attn_cross(x, x, x, x, 1, 1, 1, 1, 1, 64)
