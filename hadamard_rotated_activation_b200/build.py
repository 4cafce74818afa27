"""Build libkq.so in-tree with nvcc for sm_100a, and the _kq_call module beside it.

    python -m hadamard_rotated_activation_b200.build [--verbose]

Compiles every .cu file under csrc/ into one shared library next to this file, and
csrc/kq_call.c (C, CPython API) into an extension module of the running Python, where
there are a C compiler and Python's headers (the library needs neither).
Rebuilds only when a source or header is newer than what it is built into.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libkq.so")
CALL_SOURCE = os.path.join(CSRC, "kq_call.c")
CALL = os.path.join(HERE, "_kq_call" + sysconfig.get_config_var("EXT_SUFFIX"))

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "--expt-relaxed-constexpr",
    "-Xcompiler", "-fPIC,-fvisibility=hidden",
    "-shared",
]


def nvcc_path() -> str:
    p = shutil.which("nvcc")
    if p:
        return p
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (sources() + glob.glob(os.path.join(CSRC, "*.cuh")) +
            glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def _newer(target, deps) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(d) <= t for d in deps)


def up_to_date() -> bool:
    return _newer(LIB, _deps())


def build_call(force: bool = False):
    """The marshalling module of the decode-step calls; None (and no module) without a
    C compiler or Python's headers, which only those calls' speed needs."""
    if not force and _newer(CALL, [CALL_SOURCE, os.path.join(INCLUDE, "kq.h")]):
        return CALL
    cc = shutil.which("gcc") or shutil.which("cc")
    headers = sysconfig.get_paths()["include"]
    if not cc or not os.path.exists(os.path.join(headers, "Python.h")):
        print("kq: no " + ("Python headers" if cc else "C compiler") + ", _kq_call is not built: "
              "decode-step calls are marshalled by Python", file=sys.stderr)
        if os.path.exists(CALL):              # of an older source
            os.remove(CALL)
        return None
    tmp = f"{CALL}.{os.getpid()}.tmp"
    subprocess.run([cc, "-O2", "-Wall", "-Wextra", "-shared", "-fPIC", "-fvisibility=hidden",
                    "-I", INCLUDE, "-I", headers, "-o", tmp, CALL_SOURCE], check=True)
    os.replace(tmp, CALL)
    return CALL


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    build_call(force)
    if not force and up_to_date():
        return LIB
    cmd = [nvcc_path(), *NVCC_FLAGS, *extra, "-I", INCLUDE, "-I", CSRC,
           "-o", LIB + ".tmp", *sources()]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="--verbose" in sys.argv)
    print(LIB)
