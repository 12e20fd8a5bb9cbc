"""csrc/pycall.cpp built for CPU tensors (tests/cpu_hip), with recorders in
place of the library's functions: what the compiled calls refuse and what
they would have passed on, without a GPU."""
import ctypes
import importlib.machinery
import importlib.util
import os
import subprocess
import tempfile

import pytest

from mixed_precision_quantized_act_amd import _lib
from mixed_precision_quantized_act_amd import build as b

HERE = os.path.dirname(os.path.abspath(__file__))
NAMES = ("qlinear_bf16", "qk_norm_rope", "kv4_append", "kv4_read", "attn_kv4", "attn_cross")
ARGS = {n: _lib._SIGS[n][1] for n in NAMES}


class Calls:
    """The module `m`; `passed` holds (name, arguments) of every call that
    reached a recorder since it was last emptied."""

    def __init__(self, m):
        self.m, self.passed, self.keep = m, [], []
        for name in NAMES:
            f = ctypes.CFUNCTYPE(ctypes.c_int, *ARGS[name])(
                lambda *a, name=name: self.passed.append((name, a)) or 0)
            self.keep.append(f)
        m.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in self.keep))

    def ok(self, name, *args):
        """The arguments that the call passes on."""
        del self.passed[:]
        assert getattr(self.m, name)(*args) == 0
        (got, a), = self.passed
        assert got == name
        return a

    def refused(self, name, *args, match=None):
        del self.passed[:]
        with pytest.raises(ValueError, match=match):
            getattr(self.m, name)(*args)
        assert not self.passed


_calls = None


def calls():
    global _calls
    if _calls is None:
        pytest.importorskip("torch")
        with tempfile.TemporaryDirectory() as d:
            out = os.path.join(d, "_call.so")
            cmd = b.call_command(out)
            if cmd is None:
                pytest.skip("no host C++ compiler")
            cmd = [a for a in cmd if a != "-lc10_hip"]
            subprocess.run(cmd[:1] + ["-O0", "-I", os.path.join(HERE, "cpu_hip")] + [a for a in cmd[1:] if a != "-O2"],
                           check=True, capture_output=True)
            loader = importlib.machinery.ExtensionFileLoader("_call", out)
            m = importlib.util.module_from_spec(importlib.util.spec_from_loader("_call", loader))
            loader.exec_module(m)
        _calls = Calls(m)
    return _calls
