"""Empty tensors, which have no address: calls with nothing to do pass the
library's checks (its own functions are asked; nothing is launched)."""
import pytest

import mixed_precision_quantized_act_amd as qa
from tests._call_cpu import calls

torch = pytest.importorskip("torch")

BF, U8, INT = torch.bfloat16, torch.uint8, torch.int32


def _library(name, *args):
    """What the library answers to what the compiled call passes on."""
    return getattr(qa.lib(), name)(*calls().ok(name, *args))


@pytest.mark.parametrize("M,N", [(0, 32), (3, 0), (0, 0)])
@pytest.mark.parametrize("bias", [True, False])
def test_linear_without_rows_or_columns(M, N, bias):
    K = 64
    x, y = torch.zeros((M, K), dtype=BF), torch.zeros((M, N), dtype=BF)
    w = [torch.zeros((N, n), dtype=U8) for n in (K // 2, K // 16)]
    b = torch.zeros(N, dtype=BF) if bias else None
    assert _library("qlinear_bf16", x, *w, torch.ones(1), y, M, N, K, b, 0, 0, None, None, 0) == 0
    # the other checks are made all the same
    assert _library("qlinear_bf16", x, *w, torch.ones(1), y, M, N, 24, None, 0, 0, None, None, 0) == -2
    # (N >= 1 needs a weight)
    if N:
        assert _library("qlinear_bf16", x, None, w[1], torch.ones(1), y, M, N, K, b, 0, 0, None, None, 0) == -1


def test_heads_and_cache_without_tokens():
    H, D, page = 2, 64, 16
    e = torch.zeros((0, H * D), dtype=BF)
    w = [torch.ones(D, dtype=BF) for _ in range(4)]
    assert _library("qk_norm_rope", e, e, e, e, 0, H, H, D, 1, *w, 1e-6, 1, torch.ones((3, D // 2)),
                    torch.ones((3, D // 2)), torch.zeros(0, dtype=INT), 0) == 0
    for B, pages, entries in ((0, 4, 2), (2, 4, 2), (2, 0, 0), (2, 4, 0)):
        cache = [torch.zeros((pages, H, page, d), dtype=U8) for d in (D // 2, D // 16, D // 2, D // 16)]
        cache += [torch.ones(1), torch.ones(1), torch.zeros((B, entries), dtype=INT)]
        at = torch.zeros(B, dtype=INT)
        for T in (0, 5) if B == 0 else (0,):
            assert _library("kv4_append", e, e, *cache, at, B, T, None, 0) == 0
            assert _library("kv4_read", e, e.clone(), *cache, at, B, T, at, 0) == 0
            assert _library("attn_kv4", e, *cache, at, e, B, T, H, None, 1, None, None, 0) == 0
    s = torch.zeros((2 * 7, H * D), dtype=BF)
    assert _library("attn_cross", e, s, s, e, 2, 0, 7, H, H, D, None, None, None, None, 0) == 0
    assert _library("attn_cross", e, e, e, e, 0, 3, 0, H, H, D, torch.zeros(0, dtype=INT),
                    torch.zeros((0, 0), dtype=U8), None, None, 0) == 0
