"""Build the CUDA library in-tree: csrc/*.cu -> _build/libv4attn.so (sm_103a).

Each translation unit is compiled in parallel with nvcc; the objects are
linked into one shared library with the CUDA runtime linked statically.
Rebuilds only when a source or header is newer than the library.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import re
import shutil
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
OUT = os.path.join(HERE, "_build")
LIB = os.path.join(OUT, "libv4attn.so")
# bound-checking build (-DV4_DEBUG): indices that fail their bound record
# V4_ERR_BOUND in the device status word and the access is skipped
DEBUG_OUT = os.path.join(OUT, "debug")
DEBUG_LIB = os.path.join(DEBUG_OUT, "libv4attn_debug.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", INCLUDE, "-I", CSRC]

# Kernels that exchange registers between their warps count on what a launch starts with:
# part of the mangled name, the constant of the source that says how many.
REGISTERS = {"tree_tc.cu": ("tree_tc_kernelILb1E", "kRegsStart")}


def check_registers(src, log):
    """Refuse a build of `src` whose kernel has other registers than its split needs (log: ptxas -v)."""
    if os.path.basename(src) not in REGISTERS:
        return
    kernel, constant = REGISTERS[os.path.basename(src)]
    with open(src) as f:
        want = re.search(r"\b%s = (\d+)" % constant, f.read())
    got = re.search(r"Compiling entry function '[^']*%s(?:(?!Compiling entry).)*?Used (\d+) registers" % kernel, log, re.S)
    if not want or not got or want.group(1) != got.group(1):
        raise RuntimeError("%s: %s was compiled to %s registers, its split needs %s" % (
            os.path.basename(src), kernel, got.group(1) if got else "an unknown number of", want.group(1) if want else "?"))


def _nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def up_to_date(lib=LIB):
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(d) <= t for d in _deps())


def build(force=False, verbose=False, extra_flags=None, debug=False):
    """Compile and link the library (debug=True: the bound-checking build
    next to it); returns its path."""
    out_dir, lib = (DEBUG_OUT, DEBUG_LIB) if debug else (OUT, LIB)
    if not force and up_to_date(lib):
        return lib
    os.makedirs(out_dir, exist_ok=True)
    nvcc = _nvcc()
    extra = list(extra_flags or []) + (["-DV4_DEBUG"] if debug else [])

    def compile_one(src):
        obj = os.path.join(out_dir, os.path.basename(src)[:-3] + ".o")
        info = ["-Xptxas", "-v"] if os.path.basename(src) in REGISTERS else []
        cmd = [nvcc, *ARCH, *FLAGS, *info, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, " ".join(cmd), r.stderr))
        if verbose and r.stderr:
            print(r.stderr)
        check_registers(src, r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        objs = list(ex.map(compile_one, _sources()))
    tmp = lib + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "--cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), r.stderr))
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, debug="--debug" in sys.argv))
