"""What the compiled calls refuse, on the GPU's own tensors (the same checks
are tested one by one without a GPU in tests/test_call_*_cpu.py).  The refused
views lie in larger allocations."""
import pytest

from tests._attn import CacheCase
from tests._gpu import dev, torch

pytestmark = pytest.mark.gpu


def _qa():
    import mixed_precision_quantized_act_amd as qa
    return qa


def test_columns_of_wider_tensors_are_no_vectors():
    qa, t = _qa(), torch()
    case = CacheCase(36, 3, 2, 64, 16, [40, 40, 40])
    parts = case.device(dev)
    before = [p.clone() for p in parts]
    meta = t.full((64, 4), 3, dtype=t.int32, device="cuda")
    column = meta[:3, 1:2]
    rows = t.zeros((3, 128), dtype=t.bfloat16, device="cuda")
    o = t.full_like(rows, 7.0)
    flat = column.contiguous()
    calls = [lambda n: qa.kv4_append(rows, rows.clone(), *parts, n, 3, 1),
             lambda n: qa.kv4_read(o, t.empty_like(o), *parts, n, 3, 1),
             lambda n: qa.attn_kv4(rows, *parts, n, o, 3, 1, 2),
             lambda n: qa.attn_kv4(rows, *parts, flat, o, 3, 1, 2, q_lens=n),
             lambda n: qa.attn_cross(rows, rows, rows.clone(), o, 3, 1, 1, 2, 2, 64, k_lens=n)]
    for f in calls:
        with pytest.raises(ValueError):
            f(column)
    t.cuda.synchronize()
    assert (o == 7.0).all() and all(t.equal(a, b) for a, b in zip(parts, before))
    for f in calls:
        f(flat)
    t.cuda.synchronize()
    assert (o != 7.0).any()
