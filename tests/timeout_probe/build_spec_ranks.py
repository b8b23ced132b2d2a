"""Build test-only copies of libgdn_spec.so whose waits run out in some CTAs of
a cluster only, or in the exchanges between them (TEST INFRASTRUCTURE): the
library's own sources with switches that product builds never set, and bounded
waits of 2 ms as in build.py beside this file.

  exchange       every CTA's own arrival at its exchanges is withheld
  exchange_rank  that of the CTAs of rank 1 only
  copy_rank      the arrival at the bulk copies of the CTAs of rank 1 only
"""
import os
import subprocess

from .build import CSRC, HERE, INCLUDE, WAIT_LIMIT_NS

SPEC = os.path.join(CSRC, "spec")
SWITCHES = {"exchange": "-DGDN_TEST_WITHHOLD_EXCHANGE=-1", "exchange_rank": "-DGDN_TEST_WITHHOLD_EXCHANGE=1",
            "copy_rank": "-DGDN_TEST_WITHHOLD_COPY_RANK=1"}


def build(kind):
    lib = os.path.join(HERE, f"libgdn_spec_timeout_{kind}.so")
    deps = [os.path.join(d, f) for d in (CSRC, SPEC, INCLUDE) for f in os.listdir(d) if f.endswith((".cu", ".cuh", ".h"))]
    if os.path.exists(lib) and all(os.path.getmtime(d) <= os.path.getmtime(lib) for d in deps):
        return lib
    nvcc = "/usr/local/cuda/bin/nvcc" if os.path.exists("/usr/local/cuda/bin/nvcc") else "nvcc"
    tmp = lib + f".tmp{os.getpid()}"
    subprocess.run([nvcc, "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-std=c++17", "-shared",
                    "-Xcompiler", "-fPIC,-fvisibility=hidden", SWITCHES[kind], f"-DGDN_WAIT_LIMIT_NS={WAIT_LIMIT_NS}ull",
                    "-I", SPEC, "-I", CSRC, "-I", INCLUDE, "-o", tmp, os.path.join(SPEC, "gdn_spec_api.cu")], check=True)
    os.replace(tmp, lib)
    return lib
