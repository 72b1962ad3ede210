"""Build the HIP library libtopk.so for gfx950 (in-tree, no JIT cache).

The translation units, compiled side by side, hold the C entry points and
include their kernel headers: csrc/libtopk.hip (selection and reductions),
csrc/cache.hip (the operators on a paged key-value cache),
csrc/cache_attend.hip (its attention kernels, once for each pair of types),
csrc/sample.hip (tokens from logits) and csrc/workspace.hip (workspaces of the
last three).  The flags disable packed-FP32 instruction selection (every HIP
build in this project carries the flag), emit code for gfx950 only, and pin code
object version 5, which both the ROCm runtime in /opt/rocm and the one bundled
with PyTorch load.  They also turn off the compiler's atomic optimizer: every
atomic here is issued by one lane or targets a distinct address per lane,
and the optimizer's wave-wide combining would only add a scalar loop.

_binding.so, the native part of the Python binding (csrc/binding.cpp), is
plain C++ against PyTorch's and Python's headers; it finds libtopk.so beside
itself and PyTorch's libraries in the process that imports it.
"""
from __future__ import annotations

import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
SO = os.path.join(PKG, "libtopk.so")
BINDING = os.path.join(PKG, "_binding.so")
# Sources with their definitions: LTK_Q, LTK_C are types of include/libtopk.h.
UNITS = (("libtopk.hip",), ("cache.hip",), ("sample.hip",),
         ("workspace.hip",),
         *(("cache_attend.hip", "-DLTK_Q=%d" % q, "-DLTK_C=%d" % c)
           for q, c in ((0, 0), (0, 2), (0, 4), (1, 1), (1, 2), (1, 4))))

HIPCC_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-mcode-object-version=5",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-mllvm", "-amdgpu-atomic-optimizer-strategy=None",
    "-Wall",
]


def hipcc() -> str:
    for cand in (shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def build_libtopk(extra_flags=(), out: str = SO) -> str:
    tmp = out + ".tmp%d" % os.getpid()
    objs = ["%s.%d.o" % (tmp, i) for i in range(len(UNITS))]
    try:
        jobs = [subprocess.Popen([hipcc(), *HIPCC_FLAGS, *extra_flags, "-I",
                                  INCLUDE, "-I", CSRC, "-c",
                                  os.path.join(CSRC, u[0]), *u[1:], "-o", o])
                for u, o in zip(UNITS, objs)]
        codes = [j.wait() for j in jobs]
        for job, code in zip(jobs, codes):
            if code:
                raise subprocess.CalledProcessError(code, job.args)
        subprocess.check_call([hipcc(), "--offload-arch=gfx950", "-fPIC",
                               "-shared", *objs, "-o", tmp])
    finally:
        for o in objs:
            if os.path.exists(o):
                os.remove(o)
    os.replace(tmp, out)
    return out


def build_binding(out: str = BINDING) -> str:
    """After build_libtopk()."""
    import sysconfig
    import torch
    base = os.path.dirname(torch.__file__)
    inc = [INCLUDE, os.path.join(base, "include"),
           os.path.join(base, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"]]
    tmp = out + ".tmp%d" % os.getpid()
    subprocess.check_call(
        ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
         *(x for i in inc for x in ("-isystem" if i != INCLUDE else "-I", i)),
         os.path.join(CSRC, "binding.cpp"), "-o", tmp,
         "-L", PKG, "-l:" + os.path.basename(SO),
         "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu",
         "-lc10", "-Wl,-rpath,$ORIGIN"])
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    print(build_libtopk())
    print(build_binding())
