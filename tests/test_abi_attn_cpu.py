"""Refusals of the bf16-row linear, the head norm, the NVFP4 cache and the
attention calls, on the host: every call below fails before any launch, or
has nothing to do."""
import ctypes

import pytest

import mixed_precision_quantized_act_amd as qa

OK, EINVAL, ESHAPE, EALIGN, EALIAS = 0, -1, -2, -3, -7


def P(i):
    return ctypes.c_void_p(0x10000000 * (i + 1))     # never dereferenced


def _status(fn, args):
    return getattr(qa.lib(), fn)(*args.values())


def _expect(fn, base, changes):
    for change, want in changes:
        assert set(change) <= set(base)
        assert _status(fn, {**base, **change}) == want, (fn, change)


ODD = ctypes.c_void_p(0x10000008)


def test_qlinear_bf16_refusals():
    base = dict(x=P(0), ldx=64, w_q=P(1), w_s=P(2), w_ts=P(3), M=0, N=32, K=64, bias=None, y=P(4), ldy=32, out=0,
                epi=0, stream=None)
    _expect("qlinear_bf16", base, [
        ({}, OK), ({"M": 1, "N": 0}, OK),
        ({"x": None}, EINVAL), ({"w_q": None}, EINVAL), ({"w_s": None}, EINVAL), ({"w_ts": None}, EINVAL),
        ({"y": None}, EINVAL), ({"out": 2}, EINVAL), ({"epi": 5}, EINVAL),
        ({"M": qa.ROWS_MAX + 1}, ESHAPE), ({"M": -1}, ESHAPE), ({"K": 24}, ESHAPE), ({"K": 0}, ESHAPE),
        ({"N": -1}, ESHAPE), ({"ldx": 56}, ESHAPE), ({"ldx": 68}, ESHAPE), ({"ldx": 1 << 33}, ESHAPE),
        ({"ldy": 31}, ESHAPE), ({"K": 1 << 23, "ldx": 1 << 23}, ESHAPE),
        ({"x": ODD}, EALIGN), ({"w_q": ODD}, EALIGN), ({"bias": ctypes.c_void_p(0x10000001)}, EALIGN),
        ({"y": ctypes.c_void_p(0x10000001)}, EALIGN), ({"w_ts": ctypes.c_void_p(0x10000002)}, EALIGN),
        ({"M": 2, "y": P(0)}, EALIAS), ({"M": 2, "y": P(1)}, EALIAS), ({"M": 2, "y": P(2)}, EALIAS),
        ({"M": 2, "y": P(3)}, EALIAS), ({"M": 2, "bias": P(4)}, EALIAS)])


def test_qk_norm_rope_refusals():
    base = dict(q=P(0), ldq=256, Hq=4, k=P(1), ldk=128, Hk=2, M=0, D=64, norm=2, q_w=None, q_b=None, k_w=None,
                k_b=None, eps=1e-6, rope=1, cos=P(2), sin=P(3), P=10, pos=None, q_out=P(4), ldqo=256, k_out=P(5),
                ldko=128, stream=None)
    _expect("qk_norm_rope", base, [
        ({}, OK), ({"k": None, "Hk": 0, "k_out": None}, OK), ({"cos": None, "sin": None, "P": 0}, OK),
        ({"q": None, "k": None, "q_out": None, "k_out": None}, OK),           # no rows
        ({"M": 1, "q": None}, EINVAL), ({"M": 1, "k_out": None}, EINVAL), ({"Hk": 0}, EINVAL),
        ({"Hq": 0, "Hk": 0, "q": None, "k": None, "q_out": None, "k_out": None}, EINVAL), ({"Hq": -1}, EINVAL),
        ({"norm": 3}, EINVAL), ({"rope": 3}, EINVAL), ({"norm": 0, "q_w": P(6)}, EINVAL),
        ({"eps": -1.0}, EINVAL), ({"eps": float("nan")}, EINVAL), ({"eps": float("inf")}, EINVAL),
        ({"cos": None}, EINVAL), ({"rope": 0}, EINVAL), ({"rope": 0, "cos": None, "sin": None, "pos": P(6)}, EINVAL),
        ({"P": -1}, ESHAPE), ({"D": 24}, ESHAPE), ({"D": 0}, ESHAPE), ({"D": 272}, ESHAPE), ({"M": -1}, ESHAPE),
        ({"M": 1 << 24}, ESHAPE), ({"M": (1 << 24) - 1}, ESHAPE), ({"ldq": 248}, ESHAPE), ({"ldq": 260}, ESHAPE),
        ({"ldko": 120}, ESHAPE), ({"ldk": 1 << 32}, ESHAPE),
        ({"q": ODD}, EALIGN), ({"q_w": ODD}, EALIGN), ({"k_b": ODD}, EALIGN), ({"pos": ctypes.c_void_p(2)}, EALIGN),
        ({"cos": ctypes.c_void_p(0x10000002)}, EALIGN),
        ({"M": 4, "q_out": ctypes.c_void_p(P(0).value + 16)}, EALIAS),        # shifted on itself
        ({"M": 4, "q_out": P(0), "ldqo": 264}, EALIAS),                       # in place at another stride
        ({"M": 4, "q_out": P(1)}, EALIAS), ({"M": 4, "k_out": P(0)}, EALIAS), ({"M": 4, "k_out": P(4)}, EALIAS)])


def test_slices_of_one_buffer_do_not_overlap():
    """Columns of one row-major buffer: rows interleave, elements do not (M = 0 would skip the check)."""
    at = lambda col: ctypes.c_void_p(P(0).value + 2 * col)  # noqa: E731
    base = dict(q=at(0), ldq=512, Hq=4, k=at(256), ldk=512, Hk=2, M=4, D=64, norm=2, q_w=None, q_b=None, k_w=None,
                k_b=None, eps=1e-6, rope=3, cos=None, sin=None, P=0, pos=None, q_out=at(0), ldqo=512, k_out=at(256),
                ldko=512, stream=None)
    assert _status("qk_norm_rope", base) == EINVAL               # (the rotation's value: nothing is launched)
    base.update(rope=0)
    for change in ({"k_out": at(192)}, {"k_out": at(320)}, {"q_out": at(256 + 64)}, {"k_out": at(512)}):
        assert _status("qk_norm_rope", {**base, **change}) == EALIAS, change


def _kv(B=2, T=0):
    return dict(k=P(0), ldk=128, v=P(1), ldv=128, B=B, T=T, H=2, D=64, k_q=P(2), k_s=P(3), v_q=P(4), v_s=P(5),
                k_ts=P(6), v_ts=P(7), pages=8, page=16, table=P(8), max_pages=4, start=P(9), count=None, stream=None)


@pytest.mark.parametrize("fn", ["kv4_append", "kv4_read"])
def test_kv4_refusals(fn):
    changes = [
        ({}, OK), ({"k": None, "v": None}, OK), ({"B": 0, "T": 3, "table": None, "start": None, "k": None, "v": None}, OK),
        ({"T": 1, "k": None}, EINVAL), ({"T": 1, "v": None}, EINVAL), ({"start": None}, EINVAL), ({"k_ts": None}, EINVAL),
        ({"v_s": None}, EINVAL), ({"table": None}, EINVAL),
        ({"page": 24}, ESHAPE), ({"page": 8}, ESHAPE), ({"page": 2048}, ESHAPE), ({"page": 0}, ESHAPE),
        ({"D": 40}, ESHAPE), ({"D": 320, "ldk": 640, "ldv": 640}, ESHAPE), ({"H": 0}, ESHAPE), ({"ldk": 120}, ESHAPE),
        ({"ldv": 132}, ESHAPE), ({"T": -1}, ESHAPE), ({"B": -1}, ESHAPE), ({"pages": -1}, ESHAPE),
        ({"pages": 1 << 31}, ESHAPE), ({"pages": (1 << 31) - 1, "H": 4096, "ldk": 1 << 18, "ldv": 1 << 18}, ESHAPE),
        ({"max_pages": -1}, ESHAPE), ({"B": 1 << 12, "T": 1 << 12}, ESHAPE),
        ({"k": ODD}, EALIGN), ({"k_q": ODD}, EALIGN), ({"v_s": ODD}, EALIGN), ({"start": ctypes.c_void_p(0x10000002)}, EALIGN),
        ({"count": ctypes.c_void_p(0x10000002)}, EALIGN)]
    if fn == "kv4_append":
        changes += [({"k_q": P(3)}, EALIAS), ({"v_q": P(2)}, EALIAS), ({"T": 3, "k": P(2)}, EALIAS),
                    ({"T": 3, "v": P(5)}, EALIAS), ({"table": P(4)}, EALIAS), ({"start": P(3)}, EALIAS),
                    ({"k_ts": P(2)}, EALIAS)]
    else:
        changes += [({"T": 3, "k": P(2)}, EALIAS), ({"T": 3, "v": P(0)}, EALIAS), ({"T": 3, "v": P(8)}, EALIAS),
                    ({"T": 3, "k": P(9)}, EALIAS), ({"T": 3, "k": P(6)}, EALIAS)]
    _expect(fn, _kv(), changes)


def test_attn_kv4_refusals():
    base = dict(q=P(0), ldq=256, B=2, Lq=0, Hq=4, H=2, D=64, k_q=P(2), k_s=P(3), v_q=P(4), v_s=P(5), k_ts=P(6),
                v_ts=P(7), pages=8, page=16, table=P(8), max_pages=4, lens=P(9), q_lens=None, causal=1, scale=0.125,
                o=P(10), ldo=256, ws=None, ws_bytes=0, stream=None)
    _expect("attn_kv4", base, [
        ({}, OK), ({"q": None, "o": None}, OK),
        ({"Lq": 1, "q": None}, EINVAL), ({"Lq": 1, "o": None}, EINVAL), ({"lens": None}, EINVAL), ({"k_q": None}, EINVAL),
        ({"scale": 0.0}, EINVAL), ({"scale": -1.0}, EINVAL), ({"scale": float("nan")}, EINVAL),
        ({"scale": float("inf")}, EINVAL), ({"ws_bytes": 16}, EINVAL),
        ({"D": 80, "ldq": 320, "ldo": 320}, ESHAPE), ({"Hq": 3}, ESHAPE), ({"Hq": 0}, ESHAPE), ({"H": 0}, ESHAPE),
        ({"Lq": -1}, ESHAPE), ({"Lq": 1 << 25}, ESHAPE), ({"ldq": 248}, ESHAPE), ({"ldo": 252}, ESHAPE), ({"page": 48}, ESHAPE),
        ({"q": ODD}, EALIGN), ({"o": ODD}, EALIGN), ({"ws": ODD, "ws_bytes": 64}, EALIGN),
        ({"lens": ctypes.c_void_p(0x10000002)}, EALIGN), ({"q_lens": ctypes.c_void_p(0x10000002)}, EALIGN),
        ({"Lq": 2, "o": P(0)}, EALIAS), ({"Lq": 2, "o": P(2)}, EALIAS), ({"Lq": 2, "o": P(8)}, EALIAS),
        ({"Lq": 2, "o": P(9)}, EALIAS), ({"Lq": 2, "ws": P(0), "ws_bytes": 64}, EALIAS),
        ({"Lq": 2, "ws": P(10), "ws_bytes": 64}, EALIAS), ({"Lq": 2, "ws": P(5), "ws_bytes": 64}, EALIAS),
        ({"Lq": 2, "ws": P(9), "ws_bytes": 64}, EALIAS)])


def test_attn_cross_refusals():
    base = dict(q=P(0), ldq=256, k=P(1), ldk=128, v=P(2), ldv=128, B=2, Lq=0, Lk=5, Hq=4, Hkv=2, D=64, k_lens=None,
                mask=None, scale=0.125, o=P(3), ldo=256, ws=None, ws_bytes=0, stream=None)
    _expect("attn_cross", base, [
        ({}, OK), ({"Lk": 0, "k": None, "v": None}, OK), ({"B": 0, "Lq": 4, "q": None, "k": None, "v": None, "o": None}, OK),
        ({"k": None}, EINVAL), ({"v": None}, EINVAL), ({"Lq": 1, "q": None}, EINVAL), ({"scale": 0.0}, EINVAL),
        ({"Lk": -1}, ESHAPE), ({"Lk": 1 << 26}, ESHAPE), ({"Hkv": 3, "ldk": 192, "ldv": 192}, ESHAPE), ({"D": 32}, ESHAPE),
        ({"ldk": 120}, ESHAPE), ({"ldv": 132}, ESHAPE),
        ({"k": ODD}, EALIGN), ({"v": ODD}, EALIGN), ({"k_lens": ctypes.c_void_p(0x10000001)}, EALIGN),
        ({"Lq": 2, "o": P(0)}, EALIAS), ({"Lq": 2, "o": P(1)}, EALIAS), ({"Lq": 2, "o": P(2)}, EALIAS),
        ({"Lq": 2, "mask": P(3)}, EALIAS), ({"Lq": 2, "ws": P(1), "ws_bytes": 64}, EALIAS),
        ({"Lq": 2, "mask": P(4), "ws": P(4), "ws_bytes": 64}, EALIAS)])


def test_workspace_sizes():
    for D in (64, 128):
        for B, Lq, Hq, H, L in ((1, 1, 30, 30, 12376), (16, 1, 32, 8, 32768), (1, 1350, 30, 30, 12376), (64, 16, 64, 1, 1 << 20)):
            n = qa.attn_kv4_workspace(B, Lq, Hq, H, D, L)
            assert 0 <= n <= 32 << 20 and n == qa.attn_cross_workspace(B, Lq, L, Hq, H, D)
    for bad in ((-1, 1, 4, 2, 64, 10), (1, 1, 3, 2, 64, 10), (1, 1, 4, 2, 80, 10), (1, 1, 4, 0, 64, 10), (1, 1, 4, 2, 64, -1),
                (0, 1, 4, 2, 64, 10), (1, 0, 4, 2, 64, 10)):
        assert qa.attn_kv4_workspace(*bad) == 0
