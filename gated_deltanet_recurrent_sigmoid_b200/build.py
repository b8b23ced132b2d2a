"""Build the C-ABI libraries for sm_100a with nvcc: ``libgdn_decode.so`` (the
state update, csrc/*.cu) and ``libgdn_spec.so`` (the operators of a
speculative step around it, csrc/spec/*.cu).

The libraries are built in-tree next to this file.  ``build()`` rebuilds only
what a newer source or header asks for (or everything with ``force=True``),
and returns the path of ``libgdn_decode.so``.  ``ptxas_report()`` returns
nvcc's ``-Xptxas -v`` resource lines (registers, spills, shared memory) of
the current sources.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_NAME = "libgdn_decode.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)
SPEC_CSRC = os.path.join(CSRC, "spec")
SPEC_LIB_PATH = os.path.join(PKG, "libgdn_spec.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-shared", "-Xcompiler", "-fPIC,-fvisibility=hidden",
                     "-I", INCLUDE, "-I", CSRC, "-I", SPEC_CSRC, "--threads", "4"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libgdn_decode.so")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def spec_sources() -> list[str]:
    return sorted(glob.glob(os.path.join(SPEC_CSRC, "*.cu")))


def _deps(spec: bool = False) -> list[str]:
    shared = (glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
              + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])
    return shared + (spec_sources() + glob.glob(os.path.join(SPEC_CSRC, "*.cuh")) if spec else sources())


def _is_stale(lib: str, deps: list[str]) -> bool:
    if not os.path.exists(lib):
        return True
    built = os.path.getmtime(lib)
    return any(os.path.getmtime(d) > built for d in deps)


def stale() -> bool:
    return _is_stale(LIB_PATH, _deps())


def spec_stale() -> bool:
    return _is_stale(SPEC_LIB_PATH, _deps(spec=True))


def _compile(lib: str, srcs: list[str], verbose: bool) -> None:
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [nvcc(), *NVCC_FLAGS, "-o", tmp, *srcs]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, lib)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every CUDA source into the in-tree shared libraries."""
    if force or stale():
        _compile(LIB_PATH, sources(), verbose)
    if force or spec_stale():
        _compile(SPEC_LIB_PATH, spec_sources(), verbose)
    return LIB_PATH


def ptxas_report() -> str:
    """Registers / spills / shared memory of every kernel (nvcc -Xptxas -v)."""
    lines = []
    for srcs in (sources(), spec_sources()):
        out = os.path.join(PKG, f".ptxas_probe{os.getpid()}.so")
        try:
            res = subprocess.run([nvcc(), *NVCC_FLAGS, "-Xptxas", "-v", "-o", out, *srcs],
                                 check=True, capture_output=True, text=True)
        finally:
            if os.path.exists(out):
                os.remove(out)
        lines += [l for l in res.stderr.splitlines() if "ptxas" in l]
    return "\n".join(lines)


if __name__ == "__main__":
    if "--ptxas" in sys.argv:
        print(ptxas_report())
    else:
        print(build(force="--force" in sys.argv, verbose=True))
