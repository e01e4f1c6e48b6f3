"""Builds the in-tree shared library `_lib/libpkv.so` with nvcc for sm_100a,
and the token operators' Python binding `_lib/_tokens.so` against torch.

    python -m paged_kv_cache_frame_b200.build [--force] [--verbose]

Every CUDA and C++ source under `csrc/` is compiled to an object under
`_build/` (in parallel) and linked into one shared library with the CUDA
runtime linked statically, so loading the library needs no libcudart.so and
no GPU. The driver is reached at run time through cudaGetDriverEntryPoint.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import importlib.metadata
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_lib")
OBJ_DIR = os.path.join(ROOT, "_build")
LIB = os.path.join(OUT_DIR, "libpkv.so")
BINDING_SRC = os.path.join(HERE, "binding", "tokens.cpp")
BINDING_DEPS = [BINDING_SRC, os.path.join(HERE, "binding", "overlap.h"), os.path.join(ROOT, "include", "kv.h")]
BINDING = os.path.join(OUT_DIR, "_tokens.so")
BINDING_MADE_FOR = os.path.join(OBJ_DIR, "_tokens.for")   # the torch and Python that it was compiled against

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
COMMON = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
          f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}"]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
                  glob.glob(os.path.join(ROOT, "include", "*.h")))


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src: str, verbose: bool, ptxas_v: bool) -> str:
    obj = os.path.join(OBJ_DIR, os.path.basename(src) + ".o")
    if not _stale(obj, [src] + headers()) and not ptxas_v:
        return obj
    cmd = [nvcc(), "-c", src, "-o", obj] + ARCH + COMMON
    if src.endswith(".cpp"):
        cmd = [nvcc(), "-x", "cu", "-c", src, "-o", obj] + ARCH + COMMON
    if ptxas_v and src.endswith(".cu"):
        cmd += ["-Xptxas", "-v"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if (ptxas_v or verbose) and r.stderr:
        print(r.stderr, file=sys.stderr)
    return obj


def build(force: bool = False, verbose: bool = False, ptxas_v: bool = False) -> str:
    """Compile (if stale) and return the path of libpkv.so."""
    os.makedirs(OUT_DIR, exist_ok=True)
    os.makedirs(OBJ_DIR, exist_ok=True)
    srcs = sources()
    if not force and not ptxas_v and not _stale(LIB, srcs + headers()):
        build_binding(force, verbose)
        return LIB
    if force:
        for o in glob.glob(os.path.join(OBJ_DIR, "*.o")):
            os.remove(o)
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose, ptxas_v), srcs))
    tmp = LIB + ".tmp"
    cmd = [nvcc(), "-shared", "-o", tmp] + objs + ARCH + ["-Xcompiler", "-fPIC", "-cudart", "static",
                                                         "-ldl", "-lpthread", "-lrt"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    build_binding(force, verbose)
    return LIB


def _torch_and_python() -> str:
    try:
        torch = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        torch = "no torch"
    return f"{torch} {sys.implementation.cache_tag}"


def binding_stale() -> bool:
    """Compiled from other sources, or against another torch or Python: their
    C++ interfaces are not the same."""
    if _stale(BINDING, BINDING_DEPS) or not os.path.exists(BINDING_MADE_FOR):
        return True
    with open(BINDING_MADE_FOR) as f:
        return f.read() != _torch_and_python()


def build_binding(force: bool = False, verbose: bool = False) -> None:
    """Compile the binding (if stale) with g++; it links to libpkv.so beside it."""
    if not force and not binding_stale():
        return
    try:
        import torch
    except ImportError:   # the library itself does without; its Python objects do not
        return
    import sysconfig
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    inc = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include"), os.path.join(ROOT, "include")]
    tmp = BINDING + ".tmp"
    cmd = (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", BINDING_SRC, "-o", tmp]
           + [x for p in inc for x in ("-isystem" if p != inc[-1] else "-I", p)]
           + [f"-L{os.path.join(base, 'lib')}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda",
              f"-L{OUT_DIR}", "-lpkv", "-Wl,-rpath,$ORIGIN"])
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {BINDING_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    with open(BINDING_MADE_FOR, "w") as f:
        f.write(_torch_and_python())


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-v", action="store_true", help="print register/smem use per kernel")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose, ptxas_v=a.ptxas_v))


if __name__ == "__main__":
    main()
