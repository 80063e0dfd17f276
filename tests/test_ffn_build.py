"""What the build made of the norm and feed-forward kernels, from the library itself: no scratch
memory but in two forms, whose spilled registers are known and measured beside their kernels:
the gradient of the widest rows (read once a row), and the gradient product's exact sums with
scale rows whose stride is no multiple of 16 (read once a step of its loop).  CPU only."""

import os
import re
import shutil
import subprocess

import pytest

from block_quant_gemm_amd import build
from tests.launches import short
from tests.test_build import LLVM

#: Scratch bytes a lane.
KNOWN = {"k_norm_grad<16, 2>": 32, "k_gemm_swiglu_grad<false, true>": 128}


def test_scratch_of_the_built_kernels(tmp_path):
    tools = [os.path.join(LLVM, t) for t in ("llvm-objdump", "llvm-readelf")]
    if not all(os.path.exists(t) for t in tools):
        pytest.skip("ROCm's LLVM tools not found")
    if not os.path.exists(build.LIB):
        pytest.fail("libmxq.so is not built (run __graft_entry__.build())")
    shutil.copy(build.LIB, tmp_path / "lib.so")
    subprocess.run([tools[0], "--offloading", "lib.so"], cwd=tmp_path, check=True, capture_output=True)
    seen = {}
    for f in sorted(tmp_path.glob("lib.so.*gfx950*")):
        notes = subprocess.run([tools[1], "--notes", str(f)], check=True, capture_output=True, text=True).stdout
        for kernel in re.split(r"\n  - \.a", notes)[1:]:
            get = lambda key: re.search(rf"\.{key}: +(\S+)", kernel).group(1)
            name = short(get("name"))
            if name.startswith(("k_norm_", "k_ffn_", "k_gemm_swiglu_grad")):
                seen[name] = int(get("private_segment_fixed_size")), int(get("vgpr_spill_count"))
                assert get("uses_dynamic_stack") == "false"
    assert len(seen) >= 25 and set(KNOWN) <= set(seen), sorted(seen)
    for name, (scratch, spills) in seen.items():
        assert scratch <= KNOWN.get(name, 0) and (name in KNOWN or spills == 0), (name, scratch, spills)
