"""Build the sm_100a shared library ``libfp4q.so`` in-tree with nvcc.

    python -m fp4_micro_block_b200.build [--force]

The library is a plain C ABI (``include/fp4q.h``); nothing here links against
torch.  ``-gencode arch=compute_100a,code=sm_100a`` targets B200 only; no
fast-math, so IEEE division and square root stay correctly rounded.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libfp4q.so")
HEADER = os.path.join(ROOT, "include", "fp4q.h")


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC,-fvisibility=hidden",
    "-Xptxas", "-v",
]


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")))


TEST_LIB = os.path.join(PKG, "libfp4q_test.so")


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(s) <= t for s in sources() + [HEADER])


def build(force: bool = False, verbose: bool = False, test_hooks: bool = False,
          defines: tuple = (), out: str | None = None) -> str:
    """Builds libfp4q.so, or with test_hooks the test build libfp4q_test.so
    (bounded waits cut short and a hook that withholds one tile, so that a
    test can drive the kernels' timeout path).  `defines` (NAME=VALUE) and
    `out` build a variant of the library elsewhere, e.g.
    FP4Q_REGISTER_FWHT_MAX=64 (rotations up to 64 on the register path)."""
    lib = out or (TEST_LIB if test_hooks else LIB)
    if not force and up_to_date(lib):
        return lib
    tmp = lib + f".tmp{os.getpid()}"
    extra = (["-DFP4Q_TEST_HOOKS"] if test_hooks else []) + [f"-D{d}" for d in defines]
    units = [s for s in sources() if s.endswith(".cu")]
    objs = [f"{tmp}.{os.path.basename(u)}.o" for u in units]
    cmds = [[nvcc(), *FLAGS, *extra, "-I", os.path.join(ROOT, "include"), "-c", u, "-o", o]
            for u, o in zip(units, objs)]
    link = [nvcc(), *FLAGS[:2], "-shared", *objs, "-o", tmp]
    try:
        procs = [subprocess.Popen(c, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True) for c in cmds]
        outs = [p.communicate()[0] for p in procs]  # the translation units compile side by side
        failed = any(p.returncode != 0 for p in procs)
        if not failed:
            res = subprocess.run(link, capture_output=True, text=True)
            outs.append(res.stdout + res.stderr)
            failed = res.returncode != 0
    finally:
        for o in objs:
            if os.path.exists(o):
                os.remove(o)
    log = "".join(" ".join(c) + "\n" + t for c, t in zip(cmds + [link], outs))
    with open(os.path.join(PKG, "build_test.log" if test_hooks else "build.log"), "w") as f:
        f.write(log)
    if failed:
        raise RuntimeError("nvcc failed:\n" + log[-8000:])
    if verbose:
        print(log)
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    import argparse

    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-v", action="store_true")
    ap.add_argument("--test", action="store_true", help="the test build (libfp4q_test.so)")
    ap.add_argument("--define", action="append", default=[], help="NAME=VALUE for a library variant")
    ap.add_argument("--out", default=None, help="output path of a library variant")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.v, test_hooks=a.test, defines=tuple(a.define), out=a.out))
