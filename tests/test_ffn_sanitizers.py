"""The norm and few-token block calls' host-side argument validation under
AddressSanitizer and UndefinedBehaviorSanitizer: the sources are compiled with
both sanitizers on their host code (device code unchanged), linked into
tests/host_validation/ffn.cpp, and run where no GPU is visible.  CPU only;
the build is cached under _build/ by the digest of the sources."""

import os
import subprocess

import pytest

from tests.test_host_sanitizers import (CSRC, OUT, ROCM, ROOT, SAN, _digest, _gpu_visible, _run)

HARNESS = os.path.join(ROOT, "tests", "host_validation", "ffn.cpp")


def test_validation_under_asan_ubsan():
    if _gpu_visible():
        pytest.skip("passes fake device addresses; runs only where no GPU is visible")
    hipcc = os.path.join(ROCM, "bin", "hipcc")
    clang = os.path.join(ROCM, "llvm", "bin", "clang++")
    if not (os.path.exists(hipcc) and os.path.exists(clang)):
        pytest.skip("ROCm compilers not found")
    srcs = [os.path.join(CSRC, f) for f in ("quant.hip", "norm.hip", "ffn.hip")]
    deps = srcs + [os.path.join(CSRC, "common.h"), os.path.join(ROOT, "include", "mxq.h"), HARNESS]
    d = os.path.join(OUT, "ffn_" + _digest(deps))
    exe = os.path.join(d, "validate")
    if not os.path.exists(exe):
        os.makedirs(d, exist_ok=True)
        inc = ["-I" + os.path.join(ROOT, "include")]
        procs, objs = [], []
        for s in srcs:
            o = os.path.join(d, os.path.basename(s) + ".o")
            objs.append(o)
            procs.append(subprocess.Popen(
                [hipcc, "--offload-arch=gfx950", "-std=c++17", "-O1", "-g", "-fPIC", *inc,
                 "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", *SAN, "-c", s,
                 "-o", o], stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True))
        for p in procs:
            _, err = p.communicate()
            assert p.returncode == 0, err[-3000:]
        hobj = os.path.join(d, "validate.o")
        _run([clang, "-std=c++17", "-O1", "-g", "-D__HIP_PLATFORM_AMD__", *inc,
              "-I" + os.path.join(ROCM, "include"), *SAN, "-c", HARNESS, "-o", hobj])
        _run([clang, *SAN[:4], hobj, *objs, "-L" + os.path.join(ROCM, "lib"), "-lamdhip64",
              "-Wl,-rpath," + os.path.join(ROCM, "lib"), "-o", exe + ".tmp"])
        os.replace(exe + ".tmp", exe)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    out = (r.stdout or "") + (r.stderr or "")
    print(out)
    assert r.returncode == 0, out[-4000:]
    assert "0 failed" in out or "skipped" in out, out[-2000:]
