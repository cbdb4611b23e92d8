"""Build the in-tree C-ABI library ``libspboundary.so`` for sm_103a.

nvcc compiles each CUDA translation unit in parallel and links them into one
shared library under ``sp_boundary_norm_gb300/_build/``, and the host compiler
builds the binding's small Python module beside it.  A stamp holding a hash of
the sources and flags makes repeated builds no-ops.
"""
import concurrent.futures as cf
import hashlib
import os
import shutil
import subprocess
import sysconfig

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_build")
LIB_NAME = "libspboundary.so"
LIB_PATH = os.path.join(OUT_DIR, LIB_NAME)
MODULE_SRC = os.path.join(CSRC, "python", "tensors.cpp")
MODULE_PATH = os.path.join(OUT_DIR, "_sptensors.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
                     "-Xcompiler", "-Wall", "-I", INCLUDE, "-I", CSRC]


def _nvcc():
    for cand in (os.environ.get("CUDA_HOME", ""), "/usr/local/cuda"):
        path = os.path.join(cand, "bin", "nvcc") if cand else ""
        if path and os.path.exists(path):
            return path
    found = shutil.which("nvcc")
    if not found:
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")
    return found


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _digest(extra=()):
    h = hashlib.sha256()
    files = _sources() + [os.path.join(CSRC, f) for f in sorted(os.listdir(CSRC))
                          if f.endswith((".h", ".cuh"))]
    files.append(os.path.join(INCLUDE, "sp_boundary.h"))
    files.append(MODULE_SRC)
    for f in files:
        h.update(f.encode())
        with open(f, "rb") as fh:
            h.update(fh.read())
    h.update(" ".join(NVCC_FLAGS + list(extra)).encode())
    h.update(os.uname().machine.encode())
    h.update(torch.__version__.encode())
    return h.hexdigest()


def _build_module():
    """The binding's Python module (host code; the headers are the installed torch's)."""
    root = os.path.dirname(torch.__file__)
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-Wall",
           "-I", os.path.join(root, "include"), "-I", sysconfig.get_paths()["include"],
           "-I", os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include"),
           "-I", INCLUDE, MODULE_SRC, "-o", MODULE_PATH + ".tmp", "-L", os.path.join(root, "lib"),
           "-ltorch_python", "-ltorch", "-lc10"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"the host compiler failed for {MODULE_SRC}:\n{res.stderr}")
    os.replace(MODULE_PATH + ".tmp", MODULE_PATH)


def build_library(force=False, verbose=False, ptxas_info=False):
    """Compile (if stale) and return the path of libspboundary.so."""
    os.makedirs(OUT_DIR, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_info else []
    digest = _digest(extra)
    stamp = os.path.join(OUT_DIR, "stamp")
    if (not force and os.path.exists(LIB_PATH) and os.path.exists(MODULE_PATH)
            and os.path.exists(stamp)):
        with open(stamp) as f:
            if f.read().strip() == digest:
                return LIB_PATH
    nvcc = _nvcc()
    objs = []
    logs = {}

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc] + NVCC_FLAGS + extra + ["-c", src, "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{res.stderr}")
        return obj, res.stderr

    with cf.ThreadPoolExecutor(max_workers=min(12, os.cpu_count() or 1)) as ex:
        module = ex.submit(_build_module)
        for src, (obj, err) in zip(_sources(), ex.map(compile_one, _sources())):
            objs.append(obj)
            logs[src] = err
        module.result()
    tmp = LIB_PATH + ".tmp"
    cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + objs
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stderr}")
    os.replace(tmp, LIB_PATH)
    with open(stamp, "w") as f:
        f.write(digest)
    if verbose or ptxas_info:
        for src, err in logs.items():
            if err.strip():
                print(f"== {os.path.basename(src)}\n{err}")
    return LIB_PATH


if __name__ == "__main__":
    import sys
    print(build_library(force="--force" in sys.argv, verbose=True,
                        ptxas_info="--ptxas" in sys.argv))
