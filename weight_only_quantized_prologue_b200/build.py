"""Build libdqgemm.so in-tree with nvcc for sm_100a.

    python -m weight_only_quantized_prologue_b200.build

The library lands next to this file so it travels with the source tree.
"""

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libdqgemm.so")
# each source with the headers it includes: a source is compiled again when
# one of its own files is newer than its object
_COMMON = ["dq_handle.h", "dq_common.cuh", "dq_layout.h"]
SOURCES = {
    "dq_api.cu": _COMMON + ["dq_gemm.cuh", "dq_aux.cuh", "dq_codec.h"],
    "dq_block_api.cu": _COMMON + ["dq_block.cuh", "dq_rows.cuh", "dq_codec.h"],
    "dq_rows_api.cu": _COMMON + ["dq_rows.cuh"],
}
OBJ = os.path.join(HERE, "_build")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC,-ffp-contract=off,-O2",
    "-Xptxas", "-O3",
    "--expt-relaxed-constexpr",
]


def nvcc():
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _files(src):
    return [os.path.join(CSRC, f) for f in [src, *SOURCES[src]]] + [os.path.join(ROOT, "include", "dqgemm.h")]


def _stale(target, files):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(f) > t for f in files)


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)


def build(force=False, verbose=False, extra_flags=()):
    if not force and not _stale(LIB, [f for src in SOURCES for f in _files(src)]):
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    objs, todo = [], []
    for src in SOURCES:
        obj = os.path.join(OBJ, src.replace(".cu", ".o"))
        objs.append(obj)
        if force or _stale(obj, _files(src)):
            todo.append((src, obj))

    def compile_one(job):
        src, obj = job
        _run([nvcc(), *NVCC_FLAGS, *extra_flags, "-I", os.path.join(ROOT, "include"), "-I", CSRC,
              "-c", os.path.join(CSRC, src), "-o", obj + ".tmp"], verbose)
        os.replace(obj + ".tmp", obj)

    with ThreadPoolExecutor(len(SOURCES)) as pool:
        list(pool.map(compile_one, todo))
    _run([nvcc(), *NVCC_FLAGS, "-shared", *objs, "-o", LIB + ".tmp"], verbose)
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra_flags=("-Xptxas", "-v") if "--ptxas-v" in sys.argv else ())
