"""Build libmxq.so (the HIP kernels and their C ABI) in-tree for gfx950."""

import os
import subprocess
import sys
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SOURCES = ["csrc/quant.hip", "csrc/gemm.hip", "csrc/latent.hip", "csrc/attention.hip",
           "csrc/api.hip"]
LIB = os.path.join(PKG, "libmxq.so")
FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-fvisibility=hidden",
         # keep FP32 arithmetic off the packed-FP32 instructions
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]
# Loop-carried accumulators stay whole vectors: split into scalars, they are
# copied between the two halves of the register file in every iteration.
EXTRA_FLAGS = {s: ["-mllvm", "-amdgpu-codegenprepare-break-large-phis=0"]
               for s in ("csrc/latent.hip", "csrc/attention.hip")}


def source_digest():
    """SHA-256 of the kernel sources, the C header and the compiler's flags (identifies a build)."""
    import hashlib
    h = hashlib.sha256(repr((FLAGS, sorted(EXTRA_FLAGS.items()))).encode())
    for rel in SOURCES + ["csrc/common.h"]:
        with open(os.path.join(PKG, rel), "rb") as f:
            h.update(f.read())
    with open(os.path.join(ROOT, "include", "mxq.h"), "rb") as f:
        h.update(f.read())
    return h.hexdigest()


def hipcc():
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", "hipcc"):
        if c and (os.path.sep not in c or os.path.exists(c)):
            return c
    raise RuntimeError("hipcc not found")


def build(verbose=False):
    """Compile every source for gfx950 into block_quant_gemm_amd/libmxq.so."""
    tmp = LIB + ".tmp"
    common = [hipcc(), *FLAGS, "-I" + os.path.join(ROOT, "include")]
    with tempfile.TemporaryDirectory() as d:
        objs = [os.path.join(d, os.path.basename(s) + ".o") for s in SOURCES]
        cmds = [common + EXTRA_FLAGS.get(s, []) + ["-c", os.path.join(PKG, s), "-o", o]
                for s, o in zip(SOURCES, objs)]
        _run(cmds, verbose)
        _run([[hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp] + objs], verbose)
    os.replace(tmp, LIB)
    return LIB


def _run(cmds, verbose):
    """Runs the commands at once; raises if one fails."""
    procs = []
    for c in cmds:
        if verbose:
            print(" ".join(c), flush=True)
        procs.append(subprocess.Popen(c, stdout=subprocess.DEVNULL, stderr=subprocess.PIPE,
                                      text=True))
    errs = [p.communicate()[1] for p in procs]
    for p, err in zip(procs, errs):
        msgs = [l for l in (err or "").splitlines()
                if "packed-fp32-ops' is not a recognized feature" not in l]
        if p.returncode != 0:
            raise RuntimeError("hipcc failed:\n" + "\n".join(msgs))
        if verbose and msgs:
            print("\n".join(msgs), file=sys.stderr)


if __name__ == "__main__":
    print(build(verbose=True))
