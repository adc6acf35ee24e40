"""Build libmqv.so (the C-ABI library) in-tree with nvcc for sm_100a."""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libmqv.so")
SOURCES = ["mqv_api.cu", "mqv_layers_api.cu"]
NVCC_FLAGS = ["-std=c++17", "-O3", "-lineinfo", "-gencode", "arch=compute_100a,code=sm_100a",
              "-Xcompiler", "-fPIC,-O3", "-I", os.path.join(ROOT, "include")]


def _nvcc():
    return os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")


def _object(src):
    return os.path.join(CSRC, src[:-3] + ".o")


def _headers():
    return [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))] + \
        [os.path.join(ROOT, "include", "mqv.h")]


def _object_deps(src):
    """The files of this tree that the object was compiled from, as nvcc wrote
    them down beside it; every header where it has not, was cut off, or wrote
    them down for another place that this tree was copied from."""
    path = os.path.join(CSRC, src)
    try:
        with open(_object(src)[:-2] + ".d") as f:
            words = f.read().partition(":")[2].replace("\\\n", " ").split()
    except OSError:
        words = []
    deps = [w for w in map(os.path.realpath, words) if w.startswith(os.path.realpath(ROOT) + os.sep)]
    return deps if os.path.realpath(path) in deps else [path] + _headers()


def _stale(out, deps):
    if not os.path.exists(out) or not all(map(os.path.exists, deps)):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile what is out of date (everything with `force`), one nvcc per
    source file side by side, and link libmqv.so.  A library newer than every
    source is taken as it is, with or without the object files."""
    sources = [os.path.join(CSRC, s) for s in SOURCES]
    if not force and not _stale(LIB, sources + _headers()):
        return LIB

    def compile_one(src):
        obj = _object(src)
        if force or _stale(obj, _object_deps(src)):
            cmd = [_nvcc(), *NVCC_FLAGS, "-MD", "-MF", obj[:-2] + ".d", "-c", os.path.join(CSRC, src), "-o", obj]
            if verbose:
                cmd.insert(1, "-Xptxas=-v")
                print(" ".join(cmd), file=sys.stderr)
            subprocess.run(cmd, check=True)
        return obj

    with ThreadPoolExecutor(len(SOURCES)) as pool:
        objects = list(pool.map(compile_one, SOURCES))
    subprocess.run([_nvcc(), "-shared", *NVCC_FLAGS, *objects, "-o", LIB], check=True)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
