"""The latent attention kernels keep everything in registers: the compiler reports no
scratch memory and no spilled vector register for any of them.  They are written for
that (a spilled value costs a trip to memory in the inner loop, and a spill placed
in a block that only some lanes reach has restored a wrong address).  CPU only: it
compiles the sources for their resource report, cached by their digest."""

import os
import re
import subprocess

import pytest

from block_quant_gemm_amd import build
from tests.test_host_sanitizers import CSRC, ROOT, _digest

OUT = os.path.join(ROOT, "_build", "resources")


@pytest.mark.parametrize("name", ["latent", "attention"])
def test_no_scratch_and_no_spills(name):
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
    scratch = [int(x) for x in re.findall(r"ScratchSize \[bytes/lane\]: (\d+)", text)]
    spills = [int(x) for x in re.findall(r"[SV]GPRs Spill: (\d+)", text)]
    assert len(kernels) >= 4 and len(scratch) == len(kernels) and len(spills) == 2 * len(kernels)
    assert not any(scratch), dict(zip(kernels, scratch))
    vspills = spills[1::2]
    assert not any(vspills), dict(zip(kernels, vspills))
