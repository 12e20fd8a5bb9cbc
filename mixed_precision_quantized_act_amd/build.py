"""Build libqact.so (the HIP kernels and the C ABI) for gfx950 with hipcc, and
_call.so (the compiled Python calls) with the host compiler, where there is one
and PyTorch.

Run as ``python -m mixed_precision_quantized_act_amd.build`` or through
``__graft_entry__.build()``.  Each source compiles to its own object in
parallel (the GEMM sources hold many kernel instantiations), then one link
writes the library next to this file.
"""
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libqact.so")
CALL = os.path.join(HERE, "_call.so")
ROOT = os.path.dirname(HERE)
OBJ_DIR = os.path.join(HERE, "_build")

SOURCES = ["act_quant.hip", "qgemm.hip", "qgemm_i8.hip", "tdc.hip", "noalloc.hip", "convert_check.hip", "stage_ab.hip",
           "qgemv.hip", "qgemm_w8a8.hip", "w8a8_split.hip", "qk_norm.hip", "qk_rope.hip", "kv4.hip", "attn.hip", "attn_few.hip",
           "attn_tile.hip", "attn_tree.hip", "attn_short.hip", "abi.cpp"]

FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    # exact float32 steps in the encoders: no contraction into FMA
    "-ffp-contract=off",
    # no packed-float32 instructions in any kernel
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
]


def hipcc():
    for cand in (shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    err = "\n".join(l for l in r.stderr.splitlines() if "packed-fp32-ops" not in l)
    if r.returncode != 0:
        raise RuntimeError("compiler failed:\n" + " ".join(cmd) + "\n" + err)


def call_command(out):
    """The compiler's line for _call.so (it finds PyTorch's libraries loaded);
    None without PyTorch or a host compiler."""
    cxx, spec = shutil.which("g++") or shutil.which("c++"), importlib.util.find_spec("torch")
    if not cxx or not spec:
        return None
    torch = os.path.dirname(spec.origin)
    rocm = os.path.dirname(os.path.dirname(os.path.realpath(hipcc())))
    include = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
               os.path.join(rocm, "include"), sysconfig.get_paths()["include"]]
    return ([cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM",
             "-I", os.path.join(ROOT, "include")] + [x for d in include for x in ("-isystem", d)]
            + [os.path.join(CSRC, "pycall.cpp"), "-o", out, "-L", os.path.join(torch, "lib"),
               "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_hip"])


def build(verbose=True):
    os.makedirs(OBJ_DIR, exist_ok=True)
    cc = hipcc()
    jobs = []
    for src in SOURCES:
        obj = os.path.join(OBJ_DIR, os.path.splitext(src)[0] + ".o")
        jobs.append(([cc] + FLAGS + ["-c", os.path.join(CSRC, src), "-o", obj], obj))
    call = call_command(CALL + ".tmp")
    commands = [cmd for cmd, _ in jobs]
    if verbose:
        for cmd in ([call] if call else []) + commands:
            print(" ".join(cmd), flush=True)
    tmp = LIB + ".tmp"
    link = [cc, "--offload-arch=gfx950", "-shared", "-fPIC"] + [o for _, o in jobs] + ["-o", tmp]
    workers = max(1, min(len(commands) + 1, os.cpu_count() or 1))
    with ThreadPoolExecutor(max_workers=workers) as ex:
        # (the library does not wait for the Python calls, nor fail with them)
        called = ex.submit(_run, call) if call else None
        list(ex.map(_run, commands))
        if verbose:
            print(" ".join(link), flush=True)
        _run(link)
        # (calls that were built for another library's functions do not stay)
        if os.path.exists(CALL):
            os.remove(CALL)
        os.replace(tmp, LIB)
    if called:
        called.result()
        os.replace(CALL + ".tmp", CALL)
    else:
        print("no PyTorch or no host C++ compiler: the library alone, without _call.so", flush=True)
    return LIB


if __name__ == "__main__":
    build()
    sys.exit(0)
