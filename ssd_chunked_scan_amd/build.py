"""Compile the HIP library ``libssd.so`` (gfx950 only) in-tree with hipcc."""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libssd.so")
SOURCES = [os.path.join(CSRC, "ssd_api.hip"), os.path.join(CSRC, "gdr", "gdr_api.hip"),
           os.path.join(CSRC, "norm", "norm_api.hip")]
HEADERS = [os.path.join(ROOT, "include", "ssd.h"), os.path.join(CSRC, "ssd_device.hpp"),
           os.path.join(CSRC, "ssd_kernels.hpp"), os.path.join(CSRC, "gdr", "gdr_kernels.hpp"),
           os.path.join(CSRC, "norm", "norm_kernels.hpp")]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    # keep the compiler from forming packed-fp32 (v_pk_*_f32) instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-result",
    "-I" + os.path.join(ROOT, "include"), "-I" + CSRC,
]


# The gated delta rule's kernels hold their products' accumulators in the general
# registers; given a whole register file the compiler would put them into the
# accumulation registers and copy them out for every use.
EXTRA = {"gdr_api.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"]}


def _run(cmd, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    res = subprocess.run(cmd, capture_output=True, text=True)
    # hipcc's host pass warns that it does not know the packed-fp32 feature: harmless
    noise = "is not a recognized feature for this target"
    err = "\n".join(l for l in res.stderr.splitlines() if noise not in l)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed ({res.returncode}):\n{err}")
    if verbose and err.strip():
        print(err, file=sys.stderr)


def build_library(verbose: bool = False, extra_flags=()) -> str:
    """Compile ``libssd.so`` (the sources side by side, then one link); returns its path."""
    with tempfile.TemporaryDirectory() as obj:
        objects = [os.path.join(obj, os.path.basename(s) + ".o") for s in SOURCES]
        with ThreadPoolExecutor(len(SOURCES)) as pool:
            jobs = [pool.submit(_run, [HIPCC, *FLAGS, *EXTRA.get(os.path.basename(s), []), *extra_flags, "-c", s, "-o", o], verbose)
                    for s, o in zip(SOURCES, objects)]
            for j in jobs:
                j.result()
        tmp = LIB + ".tmp"
        _run([HIPCC, "--offload-arch=gfx950", "-fPIC", "-shared", *objects, "-o", tmp], verbose)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build_library(verbose=True))
