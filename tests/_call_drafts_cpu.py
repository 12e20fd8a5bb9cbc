"""The compiled calls of a checked step of drafted tokens for CPU tensors:
tests/_call_cpu.py's module with recorders in place of these functions too."""
import ctypes

from mixed_precision_quantized_act_amd import _lib
from tests import _call_cpu

NAMES = ("qlinear_w8a8", "qk_rope", "attn_kv4_tree", "kv4_keep")
_bound = None


def calls():
    global _bound
    c = _call_cpu.calls()
    if _bound is not c:
        for name in NAMES:
            f = ctypes.CFUNCTYPE(ctypes.c_int, *_lib._SIGS[name][1])(
                lambda *a, name=name: c.passed.append((name, a)) or 0)
            c.keep.append(f)
        c.m.bind_step(*(ctypes.cast(f, ctypes.c_void_p).value for f in c.keep[-len(NAMES):]))
        _bound = c
    return c
