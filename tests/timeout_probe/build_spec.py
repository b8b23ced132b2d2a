"""Build the test-only copy of libgdn_spec.so whose bounded waits run out
(TEST INFRASTRUCTURE): the library's own sources with the two switches that
build.py beside this file explains."""
import os
import subprocess

from .build import CSRC, HERE, INCLUDE, WAIT_LIMIT_NS

SPEC = os.path.join(CSRC, "spec")
LIB = os.path.join(HERE, "libgdn_spec_timeout.so")


def build():
    deps = [os.path.join(d, f) for d in (CSRC, SPEC, INCLUDE) for f in os.listdir(d) if f.endswith((".cu", ".cuh", ".h"))]
    if os.path.exists(LIB) and all(os.path.getmtime(d) <= os.path.getmtime(LIB) for d in deps):
        return LIB
    nvcc = "/usr/local/cuda/bin/nvcc" if os.path.exists("/usr/local/cuda/bin/nvcc") else "nvcc"
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.run([nvcc, "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-std=c++17", "-shared",
                    "-Xcompiler", "-fPIC,-fvisibility=hidden", "-DGDN_TEST_WITHHOLD_STATE_ARRIVAL",
                    f"-DGDN_WAIT_LIMIT_NS={WAIT_LIMIT_NS}ull", "-I", SPEC, "-I", CSRC, "-I", INCLUDE, "-o", tmp,
                    os.path.join(SPEC, "gdn_spec_api.cu")], check=True)
    os.replace(tmp, LIB)
    return LIB
