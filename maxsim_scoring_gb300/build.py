"""Build libmaxsim.so in-tree with nvcc for sm_103a (GB300)."""
from __future__ import annotations

import glob
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libmaxsim.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC",
    "-I", os.path.join(ROOT, "include"),
]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return (_sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")))
            + [os.path.join(ROOT, "include", "maxsim.h")])


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    nvcc = os.environ.get("NVCC", "nvcc")
    tmp = LIB + f".tmp{os.getpid()}"
    # the translation units side by side, then one link
    objects = [(src, f"{tmp}.{os.path.basename(src)}.o") for src in _sources()]
    cmds = [[nvcc, *NVCC_FLAGS, "-c", "-o", obj, src] for src, obj in objects]
    link = [nvcc, *NVCC_FLAGS, "-shared", "-o", tmp, *(obj for _, obj in objects)]
    try:
        if verbose:
            print("\n".join(" ".join(cmd) for cmd in [*cmds, link]))
        running = [subprocess.Popen(cmd) for cmd in cmds]
        codes = [p.wait() for p in running]
        for cmd, code in zip(cmds, codes):
            if code != 0:
                raise subprocess.CalledProcessError(code, cmd)
        subprocess.check_call(link)
        os.replace(tmp, LIB)
    finally:
        for _, obj in objects:
            if os.path.exists(obj):
                os.remove(obj)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
