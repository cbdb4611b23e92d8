"""Build the in-tree C-ABI library ``libspboundary.so`` for sm_103a.

nvcc compiles each CUDA translation unit in parallel and links them into one
shared library under ``sp_boundary_norm_gb300/_build/``; that needs the CUDA
toolkit alone.  Where torch is installed, the host compiler builds the binding's
small Python module beside it; a failure there is raised after the library is in
place.  A stamp of each, a hash of its sources, flags and what it is built
against, makes repeated builds no-ops.
"""
import concurrent.futures as cf
import hashlib
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

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


def _digest(files, words):
    h = hashlib.sha256()
    for f in files:
        h.update(f.encode())
        with open(f, "rb") as fh:
            h.update(fh.read())
    h.update(" ".join(words).encode())
    return h.hexdigest()


def _stamp_path(path):
    return path + ".stamp"


def _is_built(path, digest):
    if not (os.path.exists(path) and os.path.exists(_stamp_path(path))):
        return False
    with open(_stamp_path(path)) as f:
        return f.read().strip() == digest


def _put(tmp, path, digest):
    """The built file in its place, then its stamp."""
    os.replace(tmp, path)
    with open(_stamp_path(path), "w") as f:
        f.write(digest)


def _header():
    return os.path.join(INCLUDE, "sp_boundary.h")


def _torch_root():
    """Where torch is installed, or None (it is not imported)."""
    try:
        spec = importlib.util.find_spec("torch")
    except (ImportError, ValueError):
        return None
    return os.path.dirname(spec.origin) if spec is not None and spec.origin else None


def build_module(force=False):
    """Compile (if stale) and return the path of the binding's Python module, or None
    where torch, whose headers it uses, is not installed."""
    root = _torch_root()
    if root is None:
        return None
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-Wall",
           "-I", os.path.join(root, "include"), "-I", sysconfig.get_paths()["include"],
           "-I", os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include"),
           "-I", INCLUDE, MODULE_SRC, "-o", MODULE_PATH + ".tmp", "-L", os.path.join(root, "lib"),
           "-ltorch_python", "-ltorch", "-lc10"]
    # what the module's ABI depends on: the interpreter's and torch's versions
    version = os.path.join(root, "version.py")
    digest = _digest([MODULE_SRC, _header()] + [f for f in (version,) if os.path.exists(f)],
                     cmd + [sys.version, str(sysconfig.get_config_var("SOABI")),
                            os.uname().machine])
    if not force and _is_built(MODULE_PATH, digest):
        return MODULE_PATH
    os.makedirs(OUT_DIR, exist_ok=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"the host compiler failed for {MODULE_SRC}:\n{res.stderr}")
    _put(MODULE_PATH + ".tmp", MODULE_PATH, digest)
    return MODULE_PATH


def build_library(force=False, verbose=False, ptxas_info=False):
    """Compile (if stale) and return the path of libspboundary.so; the binding's module too."""
    os.makedirs(OUT_DIR, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_info else []
    headers = [os.path.join(CSRC, f) for f in sorted(os.listdir(CSRC)) if f.endswith((".h", ".cuh"))]
    digest = _digest(_sources() + headers + [_header()],
                     NVCC_FLAGS + extra + [os.uname().machine])
    logs = {}
    with cf.ThreadPoolExecutor(max_workers=min(12, os.cpu_count() or 1)) as ex:
        module = ex.submit(build_module, force)
        if force or not _is_built(LIB_PATH, digest):
            logs = _compile_library(ex, extra, digest)
    if module.result() is None and verbose:
        print("torch is not installed: the binding's module is left out")
    if verbose or ptxas_info:
        for src, err in logs.items():
            if err.strip():
                print(f"== {os.path.basename(src)}\n{err}")
    return LIB_PATH


def _compile_library(ex, extra, digest):
    """nvcc's messages by source file."""
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc] + NVCC_FLAGS + extra + ["-c", src, "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{res.stderr}")
        return obj, res.stderr

    objs, logs = [], {}
    for src, (obj, err) in zip(_sources(), ex.map(compile_one, _sources())):
        objs.append(obj)
        logs[src] = err
    tmp = LIB_PATH + ".tmp"
    res = subprocess.run([nvcc] + ARCH + ["-shared", "-o", tmp] + objs, capture_output=True,
                         text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stderr}")
    _put(tmp, LIB_PATH, digest)
    return logs


if __name__ == "__main__":
    print(build_library(force="--force" in sys.argv, verbose=True,
                        ptxas_info="--ptxas" in sys.argv))
