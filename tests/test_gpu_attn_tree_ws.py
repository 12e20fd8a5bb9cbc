"""The workspace that attn_kv4_tree asks for with few rows of a key head is the one that it
plans with: more of it changes nothing, bit by bit."""
import numpy as np
import pytest

from oracle import drafts as O
from tests._gpu import dev, torch
from tests.test_gpu_attn_tree import _qa, _trees, _ws

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,T,Hq,H", [(16, 8, 32, 8), (16, 16, 32, 8), (1, 17, 128, 128), (16, 10, 32, 8), (32, 5, 30, 6),
                                      (5, 13, 24, 8), (1, 48, 3, 3), (64, 8, 32, 8), (4, 64, 16, 16)])
def test_more_than_asked_for_changes_nothing(D, B, T, Hq, H):
    """Short streams behind tables for 32768 positions, which decide the plan."""
    qa, t = _qa(), torch()
    g = np.random.default_rng([751, D, B, T])
    page, per, cols = 64, 512, 32768
    gen = t.Generator(device="cuda").manual_seed(3)
    parts = [t.randint(0, hi, (B + 3, H, page, d), dtype=t.uint8, device="cuda", generator=gen)
             for hi, d in ((256, D // 2), (0x60, D // 16)) * 2]
    table = np.full((B, per), -1, np.int32)
    table[:, ::37] = g.integers(0, B + 3, (B, len(range(0, per, 37))))       # some positions all along it have a slot
    lens = g.integers(T, cols, B).astype(np.int32)
    lens[0] = cols
    q = t.randn((B * T, Hq * D), device="cuda", generator=gen).bfloat16()
    word, ts = dev(O.words(_trees(g, B, T, "tree"))), dev(np.array([0.01], np.float32))
    asked, out = qa.attn_kv4_tree_workspace(B, T, Hq, H, D, cols), []
    for ws in (_ws(asked) if asked else None, _ws(asked + 1000), _ws(256 << 20)):
        o = t.zeros_like(q)
        qa.attn_kv4_tree(q, *parts, ts, ts, dev(table), dev(lens), word, o, B, T, Hq, ws=ws)
        out.append(o)
    assert bool(out[0].isfinite().all()) and bool(out[0].any())
    assert t.equal(out[0], out[1]) and t.equal(out[0], out[2])
