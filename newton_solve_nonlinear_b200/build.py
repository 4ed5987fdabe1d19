"""Build the CUDA library ``libpararnn.so`` in-tree for sm_100a.

    python -m newton_solve_nonlinear_b200.build [--verbose]

Each ``csrc/*.cu`` is compiled to an object under ``_build/`` with nvcc
(``-gencode arch=compute_100a,code=sm_100a -lineinfo -O3``), then linked into
``newton_solve_nonlinear_b200/libpararnn.so`` with the CUDA runtime linked
statically.  Objects are rebuilt only when a source or header is newer.
``-Xptxas -v`` resource reports are kept in ``_build/ptxas.log``.  Kernels that
move registers between their warps rely on an exact count a thread; a compiler
that gives them another one ends the build.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import re
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libpararnn.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden", "-Xptxas", "-v",
         "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]

# registers a thread that a kernel's register split adds up to: with fewer its warps would wait for ever (the library
# refuses to launch them), with more they would not fit the card twice
EXACT_REGISTERS = {"ss_backward_kernel": 128}


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpararnn.so")


def _newest_header() -> float:
    hdrs = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(ROOT, "include", "*.h"))
    return max((os.path.getmtime(h) for h in hdrs), default=0.0)


def check_registers(log: str) -> None:
    """Raises where ptxas' report has one of EXACT_REGISTERS' kernels with another count."""
    for entry, used in re.findall(r"Compiling entry function '(\w+)'.*?Used (\d+) registers", log, re.S):
        for name, want in EXACT_REGISTERS.items():
            if name in entry and int(used) != want:
                raise RuntimeError(f"{entry} has {used} registers a thread: its split between warps needs exactly {want}")


def _compile(src: str, verbose: bool) -> tuple[str, str]:
    obj = os.path.join(BUILD, os.path.basename(src).replace(".cu", ".o"))
    if os.path.exists(obj) and os.path.getmtime(obj) >= max(os.path.getmtime(src), _newest_header()):
        return obj, ""
    cmd = [nvcc(), *ARCH, *FLAGS, "-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{res.stdout}\n{res.stderr}")
    try:
        check_registers(res.stderr)
    except RuntimeError:
        os.remove(obj)
        raise
    return obj, res.stderr


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    with cf.ThreadPoolExecutor(max_workers=min(8, len(sources))) as ex:
        results = list(ex.map(lambda s: _compile(s, verbose), sources))
    objs = [o for o, _ in results]
    logs = "".join(l for _, l in results if l)
    if logs:
        with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
            f.write(logs)
    if not os.path.exists(LIB) or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs):
        cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", LIB, *objs]
        if verbose:
            print(" ".join(cmd), flush=True)
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    return LIB


if __name__ == "__main__":
    print(build(verbose="--verbose" in sys.argv))
