"""Refusals of the 8-bit linear, the rotation by positions, the attention of
drafted tokens and the move of the kept ones, on the host: every call below
fails before any launch, or has nothing to do.  The frequencies of the
rotation, which are made on the host."""
import ctypes

import numpy as np
import pytest

import mixed_precision_quantized_act_amd as qa
from oracle import drafts as O
from tests.test_abi_attn_cpu import EALIAS, EALIGN, EINVAL, ESHAPE, ODD, OK, P, _expect

ODD4, ODD1 = ctypes.c_void_p(0x10000002), ctypes.c_void_p(0x10000001)


def test_qlinear_w8a8_refusals():
    base = dict(a_q=P(0), a_s=P(1), w_q=P(2), w_s=P(3), M=0, N=32, K=64, bias=None, y=P(4), ldy=32, out=0, epi=0,
                ws=None, ws_bytes=0, stream=None)
    _expect("qlinear_w8a8", base, [
        ({}, OK), ({"M": 1, "N": 0}, OK), ({"K": (1 << 17) - 16}, OK),
        ({"a_q": None}, EINVAL), ({"a_s": None}, EINVAL), ({"w_q": None}, EINVAL), ({"w_s": None}, EINVAL),
        ({"y": None}, EINVAL), ({"out": 2}, EINVAL), ({"epi": 5}, EINVAL), ({"ws_bytes": 16}, EINVAL),
        ({"M": -1}, ESHAPE), ({"N": -1}, ESHAPE), ({"K": 24}, ESHAPE), ({"K": 0}, ESHAPE), ({"K": 1 << 17}, ESHAPE),
        ({"M": 1 << 26}, ESHAPE), ({"ldy": 31}, ESHAPE), ({"ldy": 1 << 32}, ESHAPE),
        ({"a_q": ODD}, EALIGN), ({"w_q": ODD}, EALIGN), ({"a_s": ODD4}, EALIGN), ({"w_s": ODD4}, EALIGN),
        ({"bias": ODD1}, EALIGN), ({"y": ODD1}, EALIGN), ({"ws": ODD, "ws_bytes": 64}, EALIGN),
        ({"out": 1, "y": ODD4}, EALIGN),
        *[({"M": 2, "y": P(i)}, EALIAS) for i in range(4)], ({"M": 2, "bias": P(4)}, EALIAS),
        *[({"M": 2, "ws": P(i), "ws_bytes": 64}, EALIAS) for i in range(5)],
        ({"M": 2, "bias": P(5), "ws": P(5), "ws_bytes": 64}, EALIAS)])


def test_qk_rope_refusals():
    base = dict(q=P(0), ldq=256, Hq=4, k=P(1), ldk=128, Hk=2, M=0, D=64, R=32, rope=1, freq=P(2), scale=1.0, pos=None,
                q_out=P(4), ldqo=256, k_out=P(5), ldko=128, stream=None)
    _expect("qk_rope", base, [
        ({}, OK), ({"k": None, "Hk": 0, "k_out": None}, OK), ({"R": 64}, OK), ({"R": 16, "rope": 2}, OK),
        ({"scale": -2.0}, OK), ({"q": None, "k": None, "q_out": None, "k_out": None}, OK),
        ({"M": 1, "q": None}, EINVAL), ({"M": 1, "k_out": None}, EINVAL), ({"Hk": 0}, EINVAL), ({"freq": None}, EINVAL),
        ({"Hq": 0, "Hk": 0, "q": None, "k": None, "q_out": None, "k_out": None}, EINVAL), ({"Hq": -1}, EINVAL),
        ({"rope": 0}, EINVAL), ({"rope": 3}, EINVAL), ({"scale": float("nan")}, EINVAL), ({"scale": float("inf")}, EINVAL),
        ({"R": 0}, ESHAPE), ({"R": 8}, ESHAPE), ({"R": 40}, ESHAPE), ({"R": 80}, ESHAPE), ({"R": -16}, ESHAPE),
        ({"D": 24}, ESHAPE), ({"D": 272}, ESHAPE), ({"M": -1}, ESHAPE), ({"M": 1 << 24}, ESHAPE),
        ({"M": (1 << 24) - 1}, ESHAPE), ({"ldq": 248}, ESHAPE), ({"ldq": 260}, ESHAPE), ({"ldko": 120}, ESHAPE),
        ({"Hq": 65536, "ldq": 1 << 22, "ldqo": 1 << 22}, ESHAPE),
        ({"q": ODD}, EALIGN), ({"k_out": ODD}, EALIGN), ({"freq": ctypes.c_void_p(0x10000004)}, EALIGN),
        ({"pos": ODD4}, EALIGN),
        ({"M": 4, "q_out": ctypes.c_void_p(P(0).value + 16)}, EALIAS), ({"M": 4, "q_out": P(0), "ldqo": 264}, EALIAS),
        ({"M": 4, "q_out": P(1)}, EALIAS), ({"M": 4, "k_out": P(0)}, EALIAS), ({"M": 4, "k_out": P(4)}, EALIAS),
        ({"M": 4, "q_out": P(2)}, EALIAS), ({"M": 4, "k_out": P(2)}, EALIAS), ({"M": 4, "pos": P(4)}, EALIAS),
        ({"M": 4, "pos": P(5)}, EALIAS),
        ({"M": 4, "freq": ctypes.c_void_p(P(4).value - 32 * 4 + 8)}, EALIAS)])


def test_attn_kv4_tree_refusals():
    base = dict(q=P(0), ldq=256, B=2, Lq=0, Hq=4, H=2, D=64, k_q=P(2), k_s=P(3), v_q=P(4), v_s=P(5), k_ts=P(6),
                v_ts=P(7), pages=8, page=16, table=P(8), max_pages=4, lens=P(9), q_lens=None, tree=P(11), tree_stride=0,
                scale=0.125, o=P(10), ldo=256, ws=None, ws_bytes=0, stream=None)
    _expect("attn_kv4_tree", base, [
        ({}, OK), ({"q": None, "o": None, "tree": None}, OK), ({"tree_stride": 7}, OK),
        ({"B": 0, "Lq": 70, "tree_stride": 140}, OK),
        ({"Lq": 1, "tree": None}, EINVAL), ({"Lq": 1, "q": None}, EINVAL), ({"lens": None}, EINVAL), ({"k_q": None}, EINVAL),
        ({"scale": 0.0}, EINVAL), ({"scale": float("nan")}, EINVAL), ({"ws_bytes": 16}, EINVAL),
        ({"D": 80, "ldq": 320, "ldo": 320}, ESHAPE), ({"Hq": 3}, ESHAPE), ({"Lq": -1}, ESHAPE), ({"Lq": 1025}, ESHAPE),
        ({"Lq": 70, "tree_stride": 139}, ESHAPE), ({"Lq": 2, "tree_stride": 1}, ESHAPE), ({"tree_stride": -1}, ESHAPE),
        ({"tree_stride": 1 << 32}, ESHAPE), ({"page": 48}, ESHAPE),
        ({"tree": ctypes.c_void_p(0x10000004)}, EALIGN), ({"q": ODD}, EALIGN), ({"lens": ODD4}, EALIGN),
        ({"Lq": 2, "o": P(0)}, EALIAS), ({"Lq": 2, "o": P(2)}, EALIAS), ({"Lq": 2, "o": P(8)}, EALIAS),
        ({"Lq": 2, "o": P(9)}, EALIAS), ({"Lq": 2, "o": P(11)}, EALIAS),
        ({"Lq": 2, "ws": P(11), "ws_bytes": 64}, EALIAS), ({"Lq": 2, "ws": P(10), "ws_bytes": 64}, EALIAS),
        # the second stream's words
        ({"Lq": 2, "tree_stride": 4096, "o": ctypes.c_void_p(P(11).value + 4096 * 8)}, EALIAS)])


def test_kv4_keep_refusals():
    base = dict(k_q=P(2), k_s=P(3), v_q=P(4), v_s=P(5), B=2, T=0, H=2, D=64, pages=8, page=16, table=P(8), max_pages=4,
                start=P(9), path=P(10), count=None, stream=None)
    _expect("kv4_keep", base, [
        ({}, OK), ({"start": None, "path": None}, OK), ({"B": 0, "T": 3, "table": None, "start": None, "path": None}, OK),
        ({"T": 1, "start": None}, EINVAL), ({"T": 1, "path": None}, EINVAL), ({"k_q": None}, EINVAL),
        ({"v_s": None}, EINVAL), ({"table": None}, EINVAL),
        ({"T": -1}, ESHAPE), ({"T": 1025}, ESHAPE), ({"B": -1}, ESHAPE), ({"B": 1 << 23}, ESHAPE), ({"page": 24}, ESHAPE),
        ({"page": (1 << 30) + 1}, ESHAPE), ({"D": 40}, ESHAPE), ({"H": 0}, ESHAPE), ({"pages": 1 << 31}, ESHAPE),
        ({"k_q": ODD}, EALIGN), ({"start": ODD4}, EALIGN), ({"path": ODD4}, EALIGN), ({"count": ODD4}, EALIGN),
        ({"T": 1, "k_q": P(3)}, EALIAS), ({"T": 1, "table": P(4)}, EALIAS), ({"T": 1, "start": P(3)}, EALIAS),
        ({"T": 1, "path": P(2)}, EALIAS), ({"T": 1, "count": P(5)}, EALIAS)])


@pytest.mark.parametrize("R", [2, 4, 16, 64, 80, 128, 256])
@pytest.mark.parametrize("stretch,factor", [(0, 1.0), (0, 7.0), (1, 4.0), (2, 8.0), (3, 1.0), (3, 32.0)])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_rope_freqs(R, stretch, factor, base):
    if R == 2 and stretch == 2:
        with pytest.raises(qa.QactError):
            qa.rope_freqs(R, base, stretch, factor)
        return
    for original, fast, slow in ((4096, 32.0, 1.0), (8192, 4.0, 1.0), (1, 1.0, 1.0)):
        got, scale = qa.rope_freqs(R, base, stretch, factor, original, fast, slow)
        want, ws = O.frequencies(R, base, stretch, factor, original, fast, slow)
        # (pow, log and ten more roundings of float64; the scale rounded to float32)
        np.testing.assert_allclose(got, want, rtol=64 * 2.0 ** -53)
        assert abs(scale - ws) <= 2.0 ** -24 * ws


def test_rope_freqs_refusals():
    good = dict(R=64, base=10000.0, stretch=3, factor=4.0, original=4096, fast=32.0, slow=1.0)
    qa.rope_freqs(**good)
    inf, nan = float("inf"), float("nan")
    for change in ({"R": 63}, {"R": 0}, {"R": -2}, {"R": 65538}, {"base": 1.0}, {"base": nan}, {"base": inf}, {"factor": 0.5},
                   {"factor": nan}, {"factor": inf}, {"original": 0}, {"original": inf}, {"slow": 0.0}, {"fast": 0.5},
                   {"fast": nan}, {"stretch": 4}, {"stretch": -1}):
        with pytest.raises(qa.QactError):
            qa.rope_freqs(**{**good, **change})


def test_workspace_sizes():
    for B, Lq, Hq, H, L in ((1, 1, 30, 30, 12376), (16, 32, 32, 8, 32768), (3, 250, 30, 30, 8191)):
        assert 0 <= qa.attn_kv4_tree_workspace(B, Lq, Hq, H, 64, L) <= 32 << 20
    for bad in ((1, 1025, 4, 2, 64, 10), (-1, 1, 4, 2, 64, 10), (1, 1, 3, 2, 64, 10), (1, 1, 4, 2, 80, 10)):
        assert qa.attn_kv4_tree_workspace(*bad) == 0
    for M, N, K in ((1, 16384, 8192), (64, 7680, 1920), (17776, 5760, 1920), (300, 257, 131056), (1, 1, 16)):
        assert 0 <= qa.qlinear_w8a8_workspace(M, N, K) <= 64 << 20
    for bad in ((0, 16, 16), (16, 0, 16), (-1, 16, 16), (16, 16, 0), (16, 16, 24), (16, 16, 1 << 17), (1 << 26, 1, 16)):
        assert qa.qlinear_w8a8_workspace(*bad) == 0
