"""Build libkvb.so (the sm_100a CUDA library behind include/kvb.h) in-tree with nvcc."""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
SO = os.path.join(PKG, "libkvb.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=default"]


def _nvcc() -> str:
    for c in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found: cannot build libkvb.so")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
                  glob.glob(os.path.join(CSRC, "*.h")) + [os.path.join(ROOT, "include", "kvb.h")])


def stale() -> bool:
    if not os.path.exists(SO):
        return True
    t = os.path.getmtime(SO)
    return any(os.path.getmtime(s) > t for s in sources())


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every .cu of csrc/ (one nvcc each, side by side) and link the objects into libkvb.so."""
    if not force and not stale():
        return SO
    with tempfile.TemporaryDirectory(dir=PKG, prefix=f".build.{os.getpid()}.") as tmp:
        units = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
        objs = [os.path.join(tmp, os.path.basename(u) + ".o") for u in units]
        jobs = []
        for u, o in zip(units, objs):
            cmd = [_nvcc(), *ARCH, *FLAGS, "-c", "-o", o, u]
            if verbose:
                cmd.insert(1, "-Xptxas=-v")
                print(" ".join(cmd))
            jobs.append((cmd, subprocess.Popen(cmd)))
        codes = [(cmd, p.wait()) for cmd, p in jobs]
        for cmd, code in codes:
            if code:
                raise subprocess.CalledProcessError(code, cmd)
        so = os.path.join(tmp, "libkvb.so")
        subprocess.check_call([_nvcc(), *ARCH, "-shared", "-o", so, *objs])
        os.replace(so, SO)
    return SO


if __name__ == "__main__":
    print(build(force=True, verbose=True))
