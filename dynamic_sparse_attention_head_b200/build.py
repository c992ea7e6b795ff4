"""Builds libmsa.so (the C-ABI library) in-tree with nvcc for sm_100a, and _binding.so (torch tensors to
its calls around the layer, serving.py) with the host compiler.  The library needs neither torch nor Python's
headers; without them the binding is left out."""
from __future__ import annotations

import importlib.util
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmsa.so")
BINDING = os.path.join(HERE, "_binding.so")
BINDING_SOURCE = "binding.cpp"
BINDING_FOR = os.path.join(HERE, "_binding.for")  # the Python and torch that _binding.so was built for
SOURCES = ["plan.cu", "attn.cu", "index.cu", "estimate.cu", "lastq.cu", "permute.cu", "noalloc.cu", "selftest.cu", "recall.cu",
           "rope.cu", "kv4.cu", "kv4_attn.cu", "kv4_prompt.cu"]
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
CXX = "g++"
FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
         "--expt-relaxed-constexpr"]


def _older(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(p) > t for p in deps if os.path.exists(p))


def _header() -> str:
    return os.path.join(HERE, "..", "include", "msa.h")


def _library_stale() -> bool:
    return _older(LIB, [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != BINDING_SOURCE] + [_header()])


def _binding_for():
    """The Python and torch that a binding would be built for; None: one of them, or Python's headers, is not here."""
    if importlib.util.find_spec("torch") is None or \
            not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return None
    import torch
    return f"{sysconfig.get_config_var('SOABI')} torch {torch.__version__}"


def _binding_stale(wanted: str) -> bool:
    if _older(BINDING, [os.path.join(CSRC, BINDING_SOURCE), _header()]) or not os.path.exists(BINDING_FOR):
        return True
    with open(BINDING_FOR) as f:
        return f.read() != wanted


def _binding_command():
    from torch.utils import cpp_extension
    inc = [*cpp_extension.include_paths(), os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include"),
           sysconfig.get_paths()["include"]]
    # libmsa.so lies beside it; torch's libraries are loaded when serving.py imports torch first
    return [CXX, "-O2", "-std=c++17", "-fPIC", "-shared", "-w", *(f"-I{i}" for i in inc),
            os.path.join(CSRC, BINDING_SOURCE), "-o", BINDING, f"-L{HERE}", "-l:libmsa.so", "-Wl,-rpath,$ORIGIN",
            *(f"-L{d}" for d in cpp_extension.library_paths()), "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10", "-lc10_cuda"]


def _build_library(verbose: bool) -> None:
    objs, running = [], []
    for src in SOURCES:  # one compiler per file, side by side
        obj = os.path.join(CSRC, src.replace(".cu", ".o"))
        cmd = [NVCC, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        running.append((cmd, subprocess.Popen(cmd)))
        objs.append(obj)
    failed = [(cmd, p.returncode) for cmd, p in running if p.wait() != 0]
    if failed:
        raise subprocess.CalledProcessError(failed[0][1], failed[0][0])
    subprocess.check_call([NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", LIB, *objs])
    for o in objs:
        os.remove(o)


def build(force: bool = False, verbose: bool = False) -> str:
    if force or _library_stale():
        _build_library(verbose)
    wanted = _binding_for()
    if wanted is None:
        print("torch or Python's headers are not installed: _binding.so (serving.py) is not built", file=sys.stderr)
    elif force or _binding_stale(wanted):
        subprocess.check_call(_binding_command())
        with open(BINDING_FOR, "w") as f:
            f.write(wanted)
    return LIB


if __name__ == "__main__":
    build(force=True, verbose="-v" in sys.argv)
    for built in (LIB, BINDING):
        if os.path.exists(built):
            print(built)
