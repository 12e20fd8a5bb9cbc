"""The NVFP4 key/value cache: kv4_append writes the oracle's bytes and only
them, kv4_read gives the decoded values, rounded once to bf16."""
import numpy as np
import pytest

from oracle import attn as A
from oracle import formats as F
from tests._attn import CacheCase, bits, rng, val
from tests._gpu import dev, host, torch

pytestmark = pytest.mark.gpu


def _qa():
    import mixed_precision_quantized_act_amd as qa
    return qa


def _both(seed, B, T, H, D, page, start, count=None, pad=0, spread=1.0, **kw):
    """Append and read back on both sides; everything compared byte by byte."""
    qa, t = _qa(), torch()
    g = rng(601, seed, B, T, H, D)
    case = CacheCase(seed, B, H, D, page, [max(1, s) for s in kw.pop("lens", start)], **kw)
    width = H * D
    kv = bits(g.standard_normal((B * T, 2 * width + pad)) * spread)
    k, v = (kv[:, i * width:(i + 1) * width].reshape(B, T, H, D) for i in (0, 1))
    n = [T] * B if count is None else count
    parts = case.device(dev)
    before = [host(p).copy() for p in parts[:4]]
    d = dev(kv).view(t.bfloat16)
    st = dev(np.asarray(start, np.int32))
    ct = None if count is None else dev(np.asarray(count, np.int32))
    qa.kv4_append(d[:, :width], d[:, width:2 * width], *parts, st, B, T, count=ct)
    out = t.full((2, B * T + 1, width + 8), 7.0, dtype=t.bfloat16, device="cuda")
    qa.kv4_read(out[0], out[1], *parts, st, B, T, count=ct)
    t.cuda.synchronize()
    c = case.cache
    assert all(np.array_equal(a, b) for a, b in zip(before, (c.k_q, c.k_s, c.v_q, c.v_s)))
    c.append(k, v, start, n)
    for got, want in zip(parts[:4], (c.k_q, c.k_s, c.v_q, c.v_s)):
        np.testing.assert_array_equal(host(got), want)
    oh = host(out)
    seven = bits(np.array([7.0]))[0]
    want = np.full(oh.shape, seven)
    for b in range(B):
        for i in range(n[b]):
            if c.slot(b, start[b] + i) is not None:
                for p, x in enumerate(c.read(b, start[b] + i)):
                    want[p, b * T + i, :width] = F.f32_to_bf16_rne(x).reshape(-1)
    np.testing.assert_array_equal(oh, want)


@pytest.mark.parametrize("D", [16, 48, 64, 80, 128, 256])
@pytest.mark.parametrize("page", [16, 64])
def test_append_and_read(D, page):
    _both(1, 3, 5, 3, D, page, [0, page - 2, 3 * page + 1])


@pytest.mark.parametrize("B,T,H", [(1, 1, 1), (37, 1, 8), (1, 200, 6), (4, 33, 5)])
def test_sizes(B, T, H):
    _both(2, B, T, H, 64, 32, [(7 * b) % 90 for b in range(B)], pad=8)


def test_ragged_counts_and_positions_without_a_slot():
    # stream 0: no new tokens; 1: all; 2: a bad page in the middle; 3: past the table; 4: a
    # negative start (its first tokens have no position)
    _both(3, 5, 40, 2, 64, 16, [5, 10, 20, 45, -3], count=[0, 40, 40, 40, 9], lens=[5, 10, 20, 45, 1],
          bad=((2, 2, -1), (2, 3, 10 ** 6)))


def test_values_beyond_the_scale_and_tiny_ones():
    _both(4, 2, 9, 2, 64, 16, [3, 12], spread=40.0)
    _both(5, 2, 9, 2, 64, 16, [3, 12], spread=1e-4)


def test_zero_tokens_and_gate():
    qa, t = _qa(), torch()
    case = CacheCase(6, 2, 2, 64, 16, [5, 9])
    parts = case.device(dev)
    st = dev(np.array([5, 9], np.int32))
    e = t.empty((0, 128), dtype=t.bfloat16, device="cuda")
    qa.kv4_append(e, e, *parts, st, 2, 0)
    x = t.ones((2, 128), dtype=t.bfloat16, device="cuda")
    with qa.gate(t.zeros(1, dtype=t.uint8, device="cuda"), 1):
        qa.kv4_append(x, x, *parts, st, 2, 1)
    t.cuda.synchronize()
    assert all(np.array_equal(host(p), q) for p, q in zip(parts[:4], (
        case.cache.k_q, case.cache.k_s, case.cache.v_q, case.cache.v_s)))


def test_zero_tensor_scale():
    """A tensor scale of zero stores zeros, as the encoder's reciprocal of zero says."""
    qa, t = _qa(), torch()
    parts = [p.zero_() for p in qa.empty_kv4(3, 1, 16, 64)]
    z = t.zeros(1, device="cuda")
    table = t.tensor([[1, 2]], dtype=t.int32, device="cuda")
    st = t.zeros(1, dtype=t.int32, device="cuda")
    x = t.ones((4, 64), dtype=t.bfloat16, device="cuda")
    qa.kv4_append(x, x, *parts, z, z, table, st, 1, 4)
    out = t.full((2, 4, 64), 7.0, dtype=t.bfloat16, device="cuda")
    qa.kv4_read(out[0], out[1], *parts, z, z, table, st, 1, 4)
    assert (out == 0).all()
