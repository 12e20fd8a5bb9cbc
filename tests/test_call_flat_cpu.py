"""Vectors that the kernels read as flat memory (lengths, positions, bias,
norm weights) have to be flat: a column of a wider tensor or a broadcast
element is refused, by each of the compiled calls."""
import pytest

from tests._call_cpu import calls

torch = pytest.importorskip("torch")

B, H, D, PAGE = 4, 2, 64, 16
INT, BF = torch.int32, torch.bfloat16


def _flat_and_not(n, dtype):
    """A vector of n elements (flat in three ways), and views of n or more elements that are not flat."""
    good = [torch.zeros(n, dtype=dtype), torch.zeros(n + 3, dtype=dtype)[3:], torch.zeros((n, 1), dtype=dtype)]
    wide = torch.zeros((n, 4), dtype=dtype)
    bad = [wide[:, 1:2], wide[:, 1], torch.zeros((1, 1), dtype=dtype).expand(n, 1), torch.zeros(1, dtype=dtype).expand(n),
           torch.zeros((2, n + 1), dtype=dtype)[:, :n], torch.zeros(2 * n, dtype=dtype)[::2]]
    assert all(t.numel() >= n and not t.is_contiguous() for t in bad)
    return good, bad


def _cache():
    u8 = lambda d: torch.zeros((8, H, PAGE, d), dtype=torch.uint8)  # noqa: E731
    return [u8(D // 2), u8(D // 16), u8(D // 2), u8(D // 16), torch.ones(1), torch.ones(1),
            torch.zeros((B, 2), dtype=INT)]


def _arguments():
    """name -> (arguments, indices of the vectors with their lengths and types)"""
    rows = torch.zeros((B, H * D), dtype=BF)
    kv = lambda: [rows, rows.clone(), *_cache(), torch.zeros(B, dtype=INT), B, 1, torch.zeros(B, dtype=INT), 0]  # noqa: E731
    x, y = torch.zeros((B, 64), dtype=BF), torch.zeros((B, 32), dtype=BF)
    w = [torch.zeros((32, n), dtype=torch.uint8) for n in (32, 4)]
    norm = [torch.ones(D, dtype=BF) for _ in range(4)]
    return {
        "qlinear_bf16": ([x, *w, torch.ones(1), y, B, 32, 64, torch.zeros(32, dtype=BF), 0, 0, None, None, 0],
                         [(8, 32, BF)]),
        "qk_norm_rope": ([rows, rows.clone(), rows.clone(), rows.clone(), B, H, H, D, 1, *norm, 1e-6, 0, None, None,
                          None, 0], [(9, D, BF), (10, D, BF), (11, D, BF), (12, D, BF)]),
        "kv4_append": (kv(), [(9, B, INT), (12, B, INT)]),
        "kv4_read": (kv(), [(9, B, INT), (12, B, INT)]),
        "attn_kv4": ([rows, *_cache(), torch.zeros(B, dtype=INT), rows.clone(), B, 1, H, torch.ones(B, dtype=INT), 1,
                      None, None, 0], [(8, B, INT), (13, B, INT)]),
        "attn_cross": ([rows, rows.clone(), rows.clone(), rows.clone(), B, 1, 1, H, H, D, torch.ones(B, dtype=INT),
                        None, None, None, 0], [(10, B, INT)]),
    }


@pytest.mark.parametrize("name", ["qlinear_bf16", "qk_norm_rope", "kv4_append", "kv4_read", "attn_kv4", "attn_cross"])
def test_vectors_that_are_not_flat_are_refused(name):
    c = calls()
    args, vectors = _arguments()[name]
    c.ok(name, *args)
    for at, n, dtype in vectors:
        good, bad = _flat_and_not(n, dtype)
        for v in good:
            assert v.data_ptr() in c.ok(name, *args[:at], v, *args[at + 1:])
        for v in bad:
            c.refused(name, *args[:at], v, *args[at + 1:], match="contiguous")
