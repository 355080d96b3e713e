"""Build step for the CUDA library: nvcc, sm_103a only, in-tree.

Produces gemm_epilogue_02_gb300/libtgemm.so (git-ignored) from the translation
units csrc/tgemm_api.cu (GEMM, attention), csrc/kv_api.cu (the paged key-value
cache), csrc/page_api.cu (bounds and choice of its pages, and the pages as a
resource) and csrc/rope_api.cu (head norms with the position rotation), and its
debug build libtgemm_debug.so (-DTGEMM_DEBUG:
the device-side bounds and alignment checks of csrc/debug_checks.cuh), all
compiled in parallel.  The CUDA runtime is linked statically and the
driver's tensor-map encoder is looked up at run time, so the libraries load
(for symbol checks) on a host without a GPU driver.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRCS = [os.path.join(HERE, "csrc", f) for f in ("tgemm_api.cu", "kv_api.cu", "page_api.cu", "rope_api.cu")]
# Every header the translation units include: those of csrc and the C ABI.
DEPS = sorted(glob.glob(os.path.join(HERE, "csrc", "*.cuh")) + glob.glob(os.path.join(HERE, "csrc", "*.h"))) + [
    os.path.join(ROOT, "include", "tgemm.h")]
LIB = os.path.join(HERE, "libtgemm.so")
DEBUG_LIB = os.path.join(HERE, "libtgemm_debug.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def command(out: str, src: str, extra=()) -> list:
    """Compile one translation unit to an object file."""
    return [nvcc(), *ARCH, "-lineinfo", "-O3", "-std=c++17", "--expt-relaxed-constexpr",
            "-Xcompiler", "-fPIC", "-c", *extra, "-o", out, src]


def link_command(out: str, objects) -> list:
    return [nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", "-cudart", "static", "-o", out, *objects]


def stale(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(p) > t for p in [*SRCS, *DEPS])


def _start(cmd):
    return cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)


def _finish(jobs, verbose: bool):
    errors = []
    for cmd, proc in jobs:
        out, _ = proc.communicate()
        if proc.returncode != 0:
            errors.append("nvcc failed:\n" + " ".join(cmd) + "\n" + out)
        elif verbose and out:
            print(out)
    if errors:
        raise RuntimeError("\n".join(errors))


def build(force: bool = False, verbose: bool = False, debug: bool = True) -> str:
    """Compile libtgemm.so (and, with debug, libtgemm_debug.so) if missing or
    older than the sources, in parallel; return the release library's path."""
    libs = [lib for lib in [LIB] + ([DEBUG_LIB] if debug else []) if force or stale(lib)]
    parts = {lib: [f"{lib}.tmp{os.getpid()}.{i}.o" for i in range(len(SRCS))] for lib in libs}
    temps = [o for objs in parts.values() for o in objs] + [f"{lib}.tmp{os.getpid()}" for lib in libs]
    try:
        _finish([_start(command(obj, src, (["-DTGEMM_DEBUG"] if lib == DEBUG_LIB else []) +
                                (["-Xptxas", "-v"] if verbose else [])))
                 for lib in libs for obj, src in zip(parts[lib], SRCS)], verbose)
        _finish([_start(link_command(f"{lib}.tmp{os.getpid()}", parts[lib])) for lib in libs], verbose)
        for lib in libs:
            os.replace(f"{lib}.tmp{os.getpid()}", lib)
    finally:
        for f in temps:
            if os.path.exists(f):
                os.remove(f)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force=True, verbose="-v" in sys.argv))
