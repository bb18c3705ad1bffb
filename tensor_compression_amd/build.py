"""Build step of libkvtc: compiles the HIP sources for gfx950 with hipcc into
``tensor_compression_amd/libkvtc.so`` (in-tree, so the library travels with
the source tree).

Flags: ``-ffp-contract=off`` keeps every fused multiply-add explicit (the
kernels spell out each fma the method defines), and packed fp32 instructions
are disabled for device code.  The sources are compiled side by side.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libkvtc.so")
ARCH = os.environ.get("KVTC_OFFLOAD_ARCH", "gfx950")


def sources():
    return sorted(glob.glob(os.path.join(HERE, "csrc", "*.hip")))


def build(verbose: bool = False) -> str:
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    tmp = LIB + ".tmp"
    base = [hipcc, f"--offload-arch={ARCH}"]
    flags = ["-O3", "-std=c++17", "-fPIC", "-ffp-contract=off", "-Xclang", "-target-feature", "-Xclang",
             "-packed-fp32-ops", "-Wno-unused-result", "-I", os.path.join(ROOT, "include"), "-I",
             os.path.join(HERE, "csrc")]

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        res = subprocess.run(cmd, capture_output=True, text=True)
        errs = "\n".join(line for line in (res.stdout + res.stderr).splitlines()
                         if "packed-fp32-ops" not in line)
        if res.returncode != 0:
            raise RuntimeError(f"hipcc failed ({res.returncode}):\n{errs}")
        if verbose and errs.strip():
            print(errs, file=sys.stderr)

    with tempfile.TemporaryDirectory() as d:
        files = sources()
        objects = [os.path.join(d, os.path.basename(f) + ".o") for f in files]
        workers = max(1, min(len(files), int(os.environ.get("MAX_JOBS", os.cpu_count() or 1))))
        with ThreadPoolExecutor(workers) as pool:
            list(pool.map(lambda fo: run([*base, *flags, "-c", fo[0], "-o", fo[1]]), zip(files, objects)))
        run([*base, "-shared", "-fPIC", *objects, "-o", tmp])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
