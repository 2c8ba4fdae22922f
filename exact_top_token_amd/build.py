"""Build libhytopk.so in-tree with hipcc for gfx950.

    python -m exact_top_token_amd.build

Each HIP source is compiled to an object in ``_build/`` (in parallel), then
linked into ``exact_top_token_amd/libhytopk.so``.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libhytopk.so")
SOURCES = ["api.hip", "score.hip", "gather.hip", "radix.hip", "backward.hip", "rows.hip", "norm.hip",
           "loss.hip"]
# These keep NaN semantics: padding may hold anything, and what is not finite in a
# live entry has to show in the result.
NAN_SOURCES = ("rows.hip", "norm.hip", "loss.hip")
ARCH = os.environ.get("HYTOPK_ARCH", "gfx950")

FLAGS = [
    "-O3", "-std=c++17", f"--offload-arch={ARCH}", "-fPIC",
    # Inputs are finite by contract: without NaN semantics max(x, 0) needs no
    # canonicalising instruction in front of it.
    "-fno-honor-nans",
    # Never emit packed-fp32 VALU instructions.
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", INCLUDE, "-I", CSRC,
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def _run(cmd: list[str]) -> None:
    p = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    out = "\n".join(l for l in p.stdout.splitlines()
                    if "packed-fp32-ops" not in l and "argument unused" not in l)
    if p.returncode != 0:
        raise RuntimeError(f"command failed ({p.returncode}): {' '.join(cmd)}\n{out}")
    if out.strip():
        print(out, file=sys.stderr)


def build(verbose: bool = True) -> str:
    """Compile every HIP source and link the shared library.  Always rebuilds."""
    os.makedirs(BUILD, exist_ok=True)
    cc = hipcc()
    objs = []
    jobs = []
    for src in SOURCES:
        obj = os.path.join(BUILD, src.replace(".hip", ".o"))
        objs.append(obj)
        extra = ["-fhonor-nans"] if src in NAN_SOURCES else []
        jobs.append([cc, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj])
    workers = min(len(jobs), max(1, min(16, os.cpu_count() or 1)))
    with cf.ThreadPoolExecutor(workers) as ex:
        list(ex.map(_run, jobs))
    tmp = LIB + ".tmp"
    # -z defs: an unresolved symbol (say, a kernel whose host stub the
    # compiler dropped) fails the link instead of the first load
    _run([cc, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs,
          "-Wl,-rpath,/opt/rocm/lib", "-Wl,-z,defs"])
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build()
