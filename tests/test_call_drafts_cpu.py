"""What the compiled calls of a checked step of drafted tokens pass on and
refuse, on CPU tensors."""
import pytest

from tests._call_drafts_cpu import calls
from tests.test_call_flat_cpu import _flat_and_not

torch = pytest.importorskip("torch")

B, T, H, HQ, D, PAGE, M, N, K = 4, 3, 2, 4, 64, 16, 5, 32, 64
INT, BF, I8, F32 = torch.int32, torch.bfloat16, torch.int8, torch.float32


def _cache(scaled=True):
    u8 = lambda d: torch.zeros((8, H, PAGE, d), dtype=torch.uint8)  # noqa: E731
    ts = [torch.ones(1), torch.ones(1)] if scaled else []
    return [u8(D // 2), u8(D // 16), u8(D // 2), u8(D // 16), *ts, torch.zeros((B, 2), dtype=INT)]


def _args(name):
    rows = lambda n, h: torch.zeros((n, h * D), dtype=BF)  # noqa: E731
    return {
        "qlinear_w8a8": [torch.zeros((M, K), dtype=I8), torch.ones(M), torch.zeros((N, K), dtype=I8), torch.ones(N),
                         torch.zeros((M, N), dtype=BF), M, N, K, torch.zeros(N, dtype=BF), 0, 0, None, None, 0],
        "qk_rope": [rows(M, HQ), rows(M, H), rows(M, HQ), rows(M, H), M, HQ, H, D, 32, torch.zeros(16).double(), 2, 1.5,
                    torch.zeros(M, dtype=INT), 0],
        "attn_kv4_tree": [rows(B * T, HQ), *_cache(), torch.ones(B, dtype=INT), torch.zeros((B, T, 1), dtype=torch.long),
                          rows(B * T, HQ), B, T, HQ, torch.ones(B, dtype=INT), None, None, 0],
        "kv4_keep": [*_cache(False), torch.zeros(B, dtype=INT), torch.zeros((B, T), dtype=INT), B, T,
                     torch.ones(B, dtype=INT), 0],
    }[name]


VECTORS = {"qlinear_w8a8": [(1, M, F32), (3, N, F32), (8, N, BF)], "qk_rope": [(9, 16, torch.float64), (12, M, INT)],
           "attn_kv4_tree": [(8, B, INT), (14, B, INT)], "kv4_keep": [(5, B, INT), (9, B, INT)]}


@pytest.mark.parametrize("name", list(VECTORS))
def test_vectors(name):
    c, args = calls(), _args(name)
    c.ok(name, *args)
    for at, n, dtype in VECTORS[name]:
        good, bad = _flat_and_not(n, dtype)
        for v in good:
            assert v.data_ptr() in c.ok(name, *args[:at], v, *args[at + 1:])
        for v in bad:
            c.refused(name, *args[:at], v, *args[at + 1:], match="contiguous")
        c.refused(name, *args[:at], torch.zeros(n - 1, dtype=dtype), *args[at + 1:], match="elements")
        other = torch.float16
        c.refused(name, *args[:at], torch.zeros(n, dtype=other), *args[at + 1:], match="expected a")


def _change(name, at, value, match=None):
    args = _args(name)
    calls().refused(name, *args[:at], value, *args[at + 1:], match=match)


def test_the_linear():
    c, args = calls(), _args("qlinear_w8a8")
    a = c.ok("qlinear_w8a8", *args)
    assert a[4:7] == (M, N, K) and a[9] == N and a[13] == 0
    wide = torch.zeros((M, N + 7), dtype=BF)
    assert c.ok("qlinear_w8a8", *args[:4], wide, *args[5:])[9] == N + 7
    assert c.ok("qlinear_w8a8", *args[:4], torch.zeros((M, 40), dtype=BF), *args[5:11], 33, *args[12:])[9] == 33
    _change("qlinear_w8a8", 11, N + 1, "do not fit")                      # rows past the tensor's storage
    _change("qlinear_w8a8", 11, (1 << 63) - 1, "do not fit")
    _change("qlinear_w8a8", 5, M + 1)                                     # more rows than a_q has
    _change("qlinear_w8a8", 6, N + 1)
    _change("qlinear_w8a8", 7, K + 16)
    _change("qlinear_w8a8", 9, 1, "Float")                                # f32 output into bf16
    _change("qlinear_w8a8", 0, torch.zeros((M, 2 * K), dtype=I8)[:, :K], "contiguous")
    _change("qlinear_w8a8", 2, torch.zeros((N, 2 * K), dtype=I8)[:, ::2], "contiguous")
    _change("qlinear_w8a8", 0, torch.zeros((M, K), dtype=torch.uint8), "expected a")
    _change("qlinear_w8a8", 4, None, "expected a tensor")
    _change("qlinear_w8a8", 12, torch.zeros(64), "expected a")
    ws = torch.zeros(640, dtype=torch.uint8)
    assert c.ok("qlinear_w8a8", *args[:12], ws, args[13])[12:14] == (ws.data_ptr(), 640)
    for m, n in ((0, N), (M, 0), (0, 0)):
        got = c.ok("qlinear_w8a8", torch.zeros((m, K), dtype=I8), torch.ones(m), torch.zeros((n, K), dtype=I8),
                   torch.ones(n), torch.zeros((m, n), dtype=BF), m, n, K, None, 0, 0, None, None, 0)
        assert all(got[i] for i in (0, 1, 2, 3, 8))                       # places, if without elements


def test_the_rotation():
    c, args = calls(), _args("qk_rope")
    a = c.ok("qk_rope", *args)
    assert a[1:3] == (HQ * D, HQ) and a[7:10] == (D, 32, 2) and a[11] == 1.5
    a = c.ok("qk_rope", None, args[1], None, args[3], M, 0, *args[6:])
    assert a[0] is None and a[13] is None
    qkv = torch.zeros((M, 1024), dtype=BF)
    assert c.ok("qk_rope", qkv[:, :HQ * D], *args[1:])[1] == 1024
    _change("qk_rope", 0, qkv[:, ::2], "last dimension")
    _change("qk_rope", 0, qkv[:M - 1], "needs shape")
    _change("qk_rope", 2, qkv[:, :HQ * D - 8], "needs shape")
    _change("qk_rope", 9, torch.zeros(16), "expected a")                  # float32 frequencies
    _change("qk_rope", 9, None, "expected a tensor")
    _change("qk_rope", 8, 34, "elements")                                 # fewer frequencies than pairs
    _change("qk_rope", 8, 1 << 40, "32-bit")


def test_the_tree():
    c, args = calls(), _args("attn_kv4_tree")
    assert c.ok("attn_kv4_tree", *args)[20] == T
    one = torch.zeros((T, 1), dtype=torch.long)
    a = c.ok("attn_kv4_tree", *args[:9], one, *args[10:])
    assert a[19] == one.data_ptr() and a[20] == 0
    for bad in (torch.zeros((B - 1, T, 1), dtype=torch.long), torch.zeros((B, T, 2), dtype=torch.long),
                torch.zeros((B, T + 1, 1), dtype=torch.long), torch.zeros((B * T,), dtype=torch.long),
                torch.zeros((1, B, T, 1), dtype=torch.long)):
        _change("attn_kv4_tree", 9, bad, "tree: needs shape")
    _change("attn_kv4_tree", 9, torch.zeros((B, T, 1), dtype=INT), "expected a")
    _change("attn_kv4_tree", 9, torch.zeros((B, T, 2), dtype=torch.long)[..., :1], "contiguous")
    _change("attn_kv4_tree", 9, None, "expected a tensor")
    _change("attn_kv4_tree", 0, torch.zeros((B * T - 1, HQ * D), dtype=BF), "needs shape")
    _change("attn_kv4_tree", 7, torch.zeros((B - 1, 2), dtype=INT), "table")


def test_the_kept():
    c, args = calls(), _args("kv4_keep")
    a = c.ok("kv4_keep", *args)
    assert a[4:10] == (B, T, H, D, 8, PAGE) and a[11] == 2
    assert c.ok("kv4_keep", *args[:9], None, args[10])[14] is None
    _change("kv4_keep", 6, torch.zeros((B, T - 1), dtype=INT), "elements")
    _change("kv4_keep", 6, torch.zeros((B, 2 * T), dtype=INT)[:, :T], "contiguous")
    _change("kv4_keep", 6, torch.zeros((B, T), dtype=torch.long), "expected a")
    _change("kv4_keep", 1, torch.zeros((8, H, PAGE, 3), dtype=torch.uint8), "do not fit each other")


@pytest.mark.parametrize("name", list(VECTORS))
def test_numbers_of_arguments(name):
    with pytest.raises(TypeError):
        getattr(calls().m, name)(*_args(name)[:-1])
