"""The gradient product's host-side argument validation under AddressSanitizer and
UndefinedBehaviorSanitizer: the library's sources as tests/test_host_sanitizers.py builds them,
linked into tests/host_validation/ffn_backward.cpp, and run where no GPU is visible.  CPU only."""

import os
import subprocess

from tests.test_host_sanitizers import (CSRC, HARNESS, OUT, ROCM, ROOT, SAN, _digest, _run,
                                        test_host_validation_under_asan_ubsan as build_objects)

SRC = os.path.join(ROOT, "tests", "host_validation", "ffn_backward.cpp")


def test_gradient_product_under_asan_ubsan():
    build_objects()                                         # skips where it cannot
    srcs = [os.path.join(CSRC, f) for f in ("quant.hip", "gemm.hip", "api.hip")]
    header = os.path.join(ROOT, "include", "mxq.h")
    d = os.path.join(OUT, _digest(srcs + [os.path.join(CSRC, "common.h"), header, HARNESS]))
    exe = os.path.join(d, "ffn_backward_" + _digest([SRC]))
    if not os.path.exists(exe):
        clang, inc = os.path.join(ROCM, "llvm", "bin", "clang++"), ["-I" + os.path.join(ROOT, "include")]
        _run([clang, "-std=c++17", "-O1", "-g", "-D__HIP_PLATFORM_AMD__", *inc, "-I" + os.path.join(ROCM, "include"),
              *SAN, "-c", SRC, "-o", exe + ".o"])
        objs = [os.path.join(d, os.path.basename(s) + ".o") for s in srcs]
        _run([clang, *SAN[:4], exe + ".o", *objs, "-L" + os.path.join(ROCM, "lib"), "-lamdhip64",
              "-Wl,-rpath," + os.path.join(ROCM, "lib"), "-o", exe + ".tmp"])
        os.replace(exe + ".tmp", exe)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    out = (r.stdout or "") + (r.stderr or "")
    print(out)
    assert r.returncode == 0 and "0 failed" in out, out[-4000:]
