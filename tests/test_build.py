"""What identifies a build, and what the build made of the latent attention kernels: the
library itself says that none of them has scratch memory or a spilled vector register,
whatever sources, flags and compiler it came from.  CPU only."""

import os
import re
import shutil
import subprocess

import pytest

from block_quant_gemm_amd import build

LLVM = "/opt/rocm/llvm/bin"


def test_the_flags_are_part_of_the_digest(monkeypatch):
    before = build.source_digest()
    assert build.source_digest() == before
    monkeypatch.setattr(build, "EXTRA_FLAGS", {})
    without = build.source_digest()
    assert without != before
    monkeypatch.setattr(build, "FLAGS", build.FLAGS + ["-O2"])
    assert build.source_digest() not in (before, without)


def test_the_built_latent_kernels_use_no_scratch(tmp_path):
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
            name = re.search(r"\.symbol: +(\S+)", kernel).group(1)
            if re.search(r"k_(latent|decode|attn)_?", name):
                seen[name] = (int(get("private_segment_fixed_size")), int(get("vgpr_spill_count")),
                              get("uses_dynamic_stack"))
    assert len(seen) >= 12, sorted(seen)
    assert all(v == (0, 0, "false") for v in seen.values()), seen
