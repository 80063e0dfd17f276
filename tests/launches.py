"""What the library's norm and feed-forward calls would launch, without a GPU: runs
tests/host_validation/launches.cpp, built with the host compiler and cached under _build/
by its digest."""

import os
import re
import subprocess
from collections import namedtuple

import pytest

from block_quant_gemm_amd import mxq
from tests.test_host_sanitizers import ROCM, ROOT, _digest

SRC = os.path.join(ROOT, "tests", "host_validation", "launches.cpp")
OUT = os.path.join(ROOT, "_build", "launches")

Launch = namedtuple("Launch", "kernel grid block")


def _program():
    clang = os.path.join(ROCM, "llvm", "bin", "clang++")
    if not os.path.exists(clang):
        pytest.skip("ROCm compilers not found")
    if not os.path.exists(mxq.LIB_PATH):
        pytest.fail("libmxq.so is not built (run __graft_entry__.build())")
    exe = os.path.join(OUT, _digest([SRC, os.path.join(ROOT, "include", "mxq.h")]))
    if not os.path.exists(exe):
        os.makedirs(OUT, exist_ok=True)
        r = subprocess.run(
            [clang, "-std=c++17", "-O1", "-g", "-D__HIP_PLATFORM_AMD__", "-I" + os.path.join(ROOT, "include"),
             "-I" + os.path.join(ROCM, "include"), SRC, "-rdynamic", "-ldl", "-o", exe + ".tmp"],
            capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-3000:]
        os.replace(exe + ".tmp", exe)
    return exe


def short(name):
    """k_norm_rows<4, 1> from the mangled name of the library's kernel."""
    m = re.match(r"_ZN3mxqL?(\d+)", name)
    if not m:
        return name
    at = m.end()
    base, rest = name[at:at + int(m.group(1))], name[at + int(m.group(1)):]
    args = re.match(r"I((?:L[a-z]-?\w*?E)+)E", rest)
    if not args:
        return base
    values = [{"b0": "false", "b1": "true"}.get(a, a[1:]) for a in re.findall(r"L([a-z]\w*?)E", args.group(1))]
    return f"{base}<{', '.join(values)}>"


def run(calls):
    """(all kernels' names, [(status, [Launch])] of the calls)"""
    r = subprocess.run([_program(), mxq.LIB_PATH], input="\n".join(calls) + "\n", capture_output=True, text=True,
                       timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]
    first, *lines = r.stdout.splitlines()
    assert first.startswith("kernels;") and len(lines) == len(calls)
    out = []
    for line in lines:
        status, *launches = line.split(";")
        done = []
        for t in launches:
            name, grid, block = t.split(" ")
            done.append(Launch(short(name), *(tuple(map(int, d.split(","))) for d in (grid, block))))
        out.append((int(status), done))
    return {short(n) for n in first.split(";")[1:]}, out
