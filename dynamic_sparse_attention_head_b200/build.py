"""Builds libmsa.so (the C-ABI library) in-tree with nvcc for sm_100a, and _binding.so (torch tensors to
its calls around the layer, serving.py) with the host compiler."""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmsa.so")
BINDING = os.path.join(HERE, "_binding.so")
SOURCES = ["plan.cu", "attn.cu", "index.cu", "estimate.cu", "lastq.cu", "permute.cu", "noalloc.cu", "selftest.cu", "recall.cu",
           "rope.cu", "kv4.cu", "kv4_attn.cu", "kv4_prompt.cu"]
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
         "--expt-relaxed-constexpr"]


def _stale() -> bool:
    if not (os.path.exists(LIB) and os.path.exists(BINDING)):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(HERE, "..", "include", "msa.h")]
    return any(os.path.getmtime(p) > t for p in deps if os.path.exists(p))


def _binding_command():
    import sysconfig

    from torch.utils import cpp_extension
    inc = [*cpp_extension.include_paths(), os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include"),
           sysconfig.get_paths()["include"]]
    # libmsa.so lies beside it; torch's libraries are loaded when serving.py imports torch first
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-w", *(f"-I{i}" for i in inc),
            os.path.join(CSRC, "binding.cpp"), "-o", BINDING, f"-L{HERE}", "-l:libmsa.so", "-Wl,-rpath,$ORIGIN",
            *(f"-L{d}" for d in cpp_extension.library_paths()), "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10", "-lc10_cuda"]


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
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
    subprocess.check_call(_binding_command())
    return LIB


if __name__ == "__main__":
    build(force=True, verbose="-v" in sys.argv)
    print(LIB)
    print(BINDING)
