"""The norm's and the few-token block's kernels keep everything in registers: the compiler
reports no scratch memory for any of them but the gradient of the widest rows, whose five
spilled registers are read once a row.  CPU only: it compiles the sources for their
resource report, cached by their digest."""

import os
import re
import subprocess

import pytest

from block_quant_gemm_amd import build
from tests.test_host_sanitizers import CSRC, ROOT, _digest

OUT = os.path.join(ROOT, "_build", "resources")


@pytest.mark.parametrize("name", ["norm", "ffn"])
def test_scratch(name):
    try:
        hipcc = build.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not found")
    src = os.path.join(CSRC, name + ".hip")
    report = os.path.join(OUT, _digest([src, os.path.join(CSRC, "common.h"),
                                        os.path.join(ROOT, "include", "mxq.h")]) + ".txt")
    if not os.path.exists(report):
        os.makedirs(OUT, exist_ok=True)
        r = subprocess.run(
            [hipcc, "--offload-arch=gfx950", "--cuda-device-only", "-O3", "-std=c++17", "-fvisibility=hidden",
             "-I" + os.path.join(ROOT, "include"), "-Xclang", "-target-feature", "-Xclang",
             "-packed-fp32-ops", *build.EXTRA_FLAGS.get("csrc/" + name + ".hip", []),
             "-Rpass-analysis=kernel-resource-usage", "-c", src, "-o", os.devnull],
            capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-3000:]
        with open(report, "w") as f:
            f.write(r.stderr)
    text = open(report).read()
    kernels = re.findall(r"Function Name: (\S+)", text)
    scratch = dict(zip(kernels, map(int, re.findall(r"ScratchSize \[bytes/lane\]: (\d+)", text))))
    assert len(kernels) >= 8 and len(scratch) == len(kernels)
    widest = [k for k in kernels if "k_norm_gradILi16ELi2E" in k]
    assert len(widest) == (name == "norm")
    assert all(n <= (32 if k in widest else 0) for k, n in scratch.items()), scratch
