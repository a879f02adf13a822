"""Builds libmm.so (the HIP kernels and their C ABI) for gfx950, in-tree.

    python -m dense_bf16_gemm_amd.build

Compiler resource remarks (registers, spills, scratch, LDS per kernel) are
kept per source in ``_build/resource_usage*.txt`` next to this file.

A second library, ``libmm_fullsync.so``, is built from the same sources with
MM_DEBUG_FULL_SYNC: the slab kernel then drains every copy and waits at a
barrier before each super-step, and so do the kernels of 4-bit and 8-bit
weights before each of their steps.  It is a race check for the tests (its
results must equal libmm.so's bit for bit), never the product.
"""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmm.so")
LIB_FULLSYNC = os.path.join(HERE, "libmm_fullsync.so")
BUILD_DIR = os.path.join(HERE, "_build")
SOURCES = ["mm_api.hip", "mm_decoder.hip"]
REMARKS = os.path.join(BUILD_DIR, "resource_usage.txt")  # mm_api.hip
REMARKS_DECODER = os.path.join(BUILD_DIR, "resource_usage_decoder.txt")
ARCH = "gfx950"

HIPCC_FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    # no packed-fp32 instructions anywhere in the device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
    "-Rpass-analysis=kernel-resource-usage",
]


def hipcc() -> str:
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    cand = os.path.join(rocm, "bin", "hipcc")
    return cand if os.path.exists(cand) else "hipcc"


def _compile(source: str, obj: str, defines=()) -> list:
    return [hipcc(), *HIPCC_FLAGS, *[f"-D{d}" for d in defines], "-I", os.path.join(ROOT, "include"),
            "-c", "-o", obj, os.path.join(CSRC, source)]


def _link(out: str, objs) -> list:
    return [hipcc(), f"--offload-arch={ARCH}", "-shared", "-o", out, *objs]


def build(verbose: bool = False) -> str:
    """Builds libmm.so and the race-check libmm_fullsync.so (the hipcc runs of
    every source side by side, then the two links); returns the path of
    libmm.so.  Objects are linked in the order of SOURCES.  They and the
    compiler's output lie in a directory of this build's own, and the libraries
    and the remarks are moved into place at the end: builds at the same time
    do not read each other's files, and a failed one changes none."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    with tempfile.TemporaryDirectory(dir=BUILD_DIR) as work:
        jobs = []
        for lib, defines in ((LIB, ()), (LIB_FULLSYNC, ("MM_DEBUG_FULL_SYNC",))):
            for source in SOURCES:
                stem = os.path.join(work, os.path.splitext(source)[0] + ("" if lib == LIB else "_fullsync"))
                cmd = _compile(source, stem + ".o", defines)
                if verbose:
                    print(" ".join(cmd), flush=True)
                # compiler output to a file (a pipe could fill while the other jobs run)
                with open(stem + ".txt", "w") as f:
                    proc = subprocess.Popen(cmd, stdout=subprocess.DEVNULL, stderr=f)
                jobs.append((lib, source, stem, proc))
        failed = []
        for lib, source, stem, proc in jobs:
            if proc.wait() != 0:
                with open(stem + ".txt") as f:
                    errs = [ln for ln in f.read().splitlines() if "error" in ln]
                failed.append(f"hipcc failed for {source} ({os.path.basename(lib)}):\n" + "\n".join(errs[:40]))
        if failed:
            raise RuntimeError("\n".join(failed))
        linked = []
        for lib in (LIB, LIB_FULLSYNC):
            out = os.path.join(work, os.path.basename(lib))
            cmd = _link(out, [stem + ".o" for (of, _, stem, _) in jobs if of == lib])
            if verbose:
                print(" ".join(cmd), flush=True)
            subprocess.run(cmd, check=True)
            linked.append((out, lib))
        for lib, source, stem, _ in jobs:
            if lib == LIB:
                linked.append((stem + ".txt", REMARKS if source == "mm_api.hip" else REMARKS_DECODER))
        for made, place in linked:
            os.replace(made, place)
    return LIB


def resource_usage(path: str = REMARKS):
    """Parses the resource remarks into {kernel: {field: int}} (True / False
    fields, such as "Dynamic Stack", as 1 / 0)."""
    out = {}
    cur = None
    with open(path) as f:
        for line in f:
            if "remark:" not in line:
                continue
            body = line.split("remark:", 1)[1].strip()
            body = body.replace("[-Rpass-analysis=kernel-resource-usage]", "").strip()
            if body.startswith("Function Name:"):
                cur = body.split(":", 1)[1].strip()
                out[cur] = {}
            elif cur is not None and ":" in body:
                key, val = body.rsplit(":", 1)
                val = {"True": "1", "False": "0"}.get(val.strip(), val.strip())
                try:
                    out[cur][key.strip()] = int(val)
                except ValueError:
                    pass
    return out


if __name__ == "__main__":
    print(build(verbose=True))
    sys.exit(0)
