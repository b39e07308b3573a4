"""Build the gfx950 library in-tree: ``python sparse_spatial_hashing_amd/csrc/build.py``.

A standalone script (the package itself refuses to import without the library).

Flags: -O3, no fast-math (binning must be IEEE fp32), no FMA contraction,
packed-FP32 instructions disabled, position-independent shared object.
"""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

CSRC = os.path.dirname(os.path.abspath(__file__))
HERE = os.path.dirname(CSRC)
ROOT = os.path.dirname(HERE)
SOURCES = [os.path.join(CSRC, f) for f in ("voxelize.hip", "spherical.hip", "embed.hip", "scan.hip",
                                           "attend.hip")]
# compiled once per element type and padded head width
ATTENTION = os.path.join(CSRC, "attend_kernels.hip")
UNITS = [(s, []) for s in SOURCES] + [(ATTENTION, [f"-DATT_WIDTH={w}", f"-DATT_F16={f}"])
                                      for w in (32, 64, 128) for f in (0, 1)]
SOURCE = SOURCES[0]
HEADER = os.path.join(ROOT, "include", "voxelize.h")
LIBRARY = os.path.join(HERE, "libvoxelize.so")
ARCH = os.environ.get("VOX_OFFLOAD_ARCH", "gfx950")

HIPCC_FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-ffp-contract=off", "-fno-fast-math",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-fPIC", "-Wall",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", "hipcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    raise RuntimeError("hipcc not found")


def _run(cmd, quiet: bool) -> None:
    res = subprocess.run(cmd, capture_output=True, text=True)
    noise = "packed-fp32-ops"
    msgs = "\n".join(l for l in (res.stdout + res.stderr).splitlines() if noise not in l)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed ({res.returncode}):\n{msgs}")
    if msgs.strip() and not quiet:
        print(msgs, file=sys.stderr)


def build(output: str = LIBRARY, quiet: bool = False) -> str:
    """Compile every unit (a few at a time) and link the library."""
    tmp = output + ".tmp"
    include = os.path.dirname(HEADER)
    with tempfile.TemporaryDirectory(prefix="ssh_build_") as work:
        objects = [os.path.join(work, f"{i}.o") for i in range(len(UNITS))]
        with ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as pool:
            jobs = [pool.submit(_run, [hipcc(), *HIPCC_FLAGS, *defines, "-I", include, "-c", source,
                                       "-o", obj], quiet)
                    for (source, defines), obj in zip(UNITS, objects)]
            for job in jobs:
                job.result()
        _run([hipcc(), f"--offload-arch={ARCH}", "-fPIC", "-shared", "-o", tmp, *objects], quiet)
    os.replace(tmp, output)
    return output


if __name__ == "__main__":
    print(build())
