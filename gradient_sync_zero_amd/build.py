"""Builds libgsz.so in-tree with hipcc for gfx950."""
from __future__ import annotations

import os
import subprocess

_HERE = os.path.dirname(os.path.abspath(__file__))
_ROOT = os.path.dirname(_HERE)

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
LIB = os.path.join(_HERE, "libgsz.so")
# The same sources with the test hooks of include/gsz_test.h compiled in.
TEST_LIB = os.path.join(_HERE, "libgsz_test.so")

# -ffp-contract=off: the AdamW update and the fp32 reduction must keep one
# rounding per operation (no fused multiply-add).  Packed fp32 instructions are
# switched off.  Division and sqrt stay IEEE correctly rounded (clang's HIP
# default); fp32 denormals are kept.
FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
         "-ffp-contract=off", "-fno-fast-math",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-Wall", "-Wno-unused-result",
         "-I", os.path.join(_ROOT, "include"), "-I", os.path.join(_HERE, "csrc"),
         "-I", os.path.join(_HERE, "matrix")]
LINK_FLAGS = ["--offload-arch=gfx950", "-fPIC", "-shared", "-Wl,-rpath,/opt/rocm/lib"]
# csrc/ holds the step; layers/ the embedding, dropout and position bias kernels around it,
# optim/ the orthogonalising optimizer, matrix/ what that takes from the matrix cores (the
# step's counter summaries are keyed to csrc/ alone).
SOURCES = ["csrc/plan.cpp", "csrc/gsz_step.hip", "layers/gsz_layers.hip", "layers/gsz_relpos.hip",
           "optim/gsz_muon.hip"]
# The sources that hold test hooks; the others' objects serve both libraries.
HOOKED = ("csrc/plan.cpp", "csrc/gsz_step.hip")


def build(verbose: bool = False) -> str:
    """Builds libgsz.so and libgsz_test.so: every source of both side by side, then the links."""
    import tempfile

    def run(cmds):
        if verbose:
            print("\n".join(" ".join(c) for c in cmds), flush=True)
        procs = [subprocess.Popen(c, cwd=_HERE) for c in cmds]
        failed = [c for c, p in zip(cmds, procs) if p.wait() != 0]
        if failed:
            raise subprocess.CalledProcessError(1, failed[0])

    with tempfile.TemporaryDirectory(prefix="_build", dir=_HERE) as tmp:
        compiles, links = [], []
        for out, hooks in ((LIB, False), (TEST_LIB, True)):
            objs = []
            for src in SOURCES:
                own = hooks and src in HOOKED
                objs.append(os.path.join(tmp, ("hooks_" if own else "") + os.path.basename(src) + ".o"))
                if own or not hooks:
                    compiles.append([HIPCC, *FLAGS, *(["-DGSZ_TEST_HOOKS"] if own else []), "-c", src, "-o", objs[-1]])
            links.append([HIPCC, *LINK_FLAGS, *objs, "-o", out + ".tmp"])
        run(compiles)
        run(links)
    for out in (LIB, TEST_LIB):
        os.replace(out + ".tmp", out)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
