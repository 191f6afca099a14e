"""Build liblf_hsa.so in place: every kernel compiled for sm_100a with nvcc."""
from __future__ import annotations

import os
import re
import subprocess
import sys

_HERE = os.path.dirname(os.path.abspath(__file__))
_ROOT = os.path.dirname(_HERE)
SOURCES = ["lf_api.cu", "lf_pool.cu", "lf_select.cu", "lf_ivf.cu", "lf_quant.cu", "lf_attn.cu",
           "lf_attn_bwd.cu", "lf_rope.cu", "lf_norm.cu",
           "lf_norm_bwd.cu"]
HEADERS = ["lf_device.cuh", "lf_internal.h", "lf_score.cuh", "lf_types.cuh", "lf_attn_bwd.h", "lf_rope.h",
           "lf_norm.h", "lf_norm_rows.cuh"]
LIB = os.path.join(_HERE, "liblf_hsa.so")
OBJ_DIR = os.path.join(_HERE, "_build")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC,-O2,-fvisibility=hidden",
    "--expt-relaxed-constexpr",
]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(_HERE, "csrc", f) for f in SOURCES + HEADERS]
    deps.append(os.path.join(_ROOT, "include", "lf_hsa.h"))
    deps.append(os.path.abspath(__file__))
    return any(os.path.getmtime(p) > t for p in deps)


def _depends(path: str) -> set:
    """The file and the library's own headers that it includes."""
    found, todo = set(), [path]
    while todo:
        p = todo.pop()
        if p in found:
            continue
        found.add(p)
        with open(p) as f:
            for name in re.findall(r'^#include "([^"]+)"', f.read(), re.M):
                at = [os.path.join(d, name) for d in (os.path.dirname(path), os.path.join(_ROOT, "include"))]
                todo += [q for q in at if os.path.exists(q)]
    return found


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compiles the stale translation units in parallel (objects kept under _build/) and links them."""
    if not force and not ptxas_info and not _stale():
        return LIB
    os.makedirs(OBJ_DIR, exist_ok=True)
    nvcc = _nvcc()
    objs, running = [], []
    for f in SOURCES:
        src, obj = os.path.join(_HERE, "csrc", f), os.path.join(OBJ_DIR, f + ".o")
        objs.append(obj)
        fresh = os.path.exists(obj) and all(os.path.getmtime(p) < os.path.getmtime(obj)
                                            for p in _depends(src) | {os.path.abspath(__file__)})
        if fresh and not force and not ptxas_info:
            continue
        cmd = [nvcc, *NVCC_FLAGS, "-I", os.path.join(_ROOT, "include"), "-c", "-o", obj + ".tmp", src]
        if ptxas_info:
            cmd.insert(1, "-Xptxas=-v")
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        running.append((subprocess.Popen(cmd), obj, cmd))
    failed = [cmd for p, _, cmd in running if p.wait() != 0]
    if failed:
        raise subprocess.CalledProcessError(1, failed[0])
    for _, obj, _ in running:
        os.replace(obj + ".tmp", obj)
    tmp = LIB + ".tmp"
    subprocess.run([nvcc, *NVCC_FLAGS, "-shared", "-cudart", "static", "-o", tmp, *objs, "-ldl", "-lrt", "-lpthread"],
                   check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True, ptxas_info="-v" in sys.argv))
