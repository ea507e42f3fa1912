"""Build libvsa.so (the C-ABI library) in-tree with nvcc for sm_100a.

    python -m block_sparse_video_tile_b200.build [--force]

The shared library is written next to this file, so it travels with the
source tree.  No GPU is needed to build (nvcc cross-compiles).
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
COMMON = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]
OBJ = os.path.join(PKG, "_build")          # objects and their dependency lists

TARGETS = {
    "libvsa.so": ["libvsa.cu", "norm_rope.cu", "window.cu"],   # the product: C ABI of include/vsa.h
    "libvsa_diag.so": ["vsa_diag.cu"],                          # bring-up checks used by the tests only
}


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libvsa")
    return cand


def _stale(obj: str, dep: str) -> bool:
    """Whether an object is older than a file it was compiled from (nvcc's dependency list)."""
    if not (os.path.exists(obj) and os.path.exists(dep)):
        return True
    with open(dep) as f:
        files = f.read().replace("\\\n", " ").split(":", 1)[-1].split()
    made = os.path.getmtime(obj)
    return any(not os.path.exists(p) or os.path.getmtime(p) > made for p in files + [__file__])


def _finish(what: str, p: subprocess.Popen, verbose: bool) -> None:
    out, _ = p.communicate()
    if p.returncode != 0:
        raise RuntimeError(f"nvcc failed for {what}:\n{out}")
    if verbose and out:
        print(out, flush=True)


def _run(cmd, verbose: bool) -> subprocess.Popen:
    if verbose:
        print(" ".join(cmd), flush=True)
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)


def build(force: bool = False, verbose: bool = False, extra=()) -> list:
    """Compile every target (the sources side by side, only those that changed) and link;
    returns the paths of the built libraries."""
    os.makedirs(OBJ, exist_ok=True)
    running, out = [], []
    for srcs in TARGETS.values():
        for src in srcs:
            obj = os.path.join(OBJ, src + ".o")
            dep = obj + ".d"
            if force or _stale(obj, dep):
                running.append((src, obj, _run([_nvcc(), *ARCH, *COMMON, *extra, "-c", os.path.join(CSRC, src), "-MD",
                                                "-MF", dep, "-o", obj + ".tmp"], verbose)))
    try:
        for src, obj, p in running:
            _finish(src, p, verbose)
            os.replace(obj + ".tmp", obj)
    finally:
        for _, _, p in running:
            if p.poll() is None:
                p.kill()
                p.wait()
    for lib, srcs in TARGETS.items():
        dst, objs = os.path.join(PKG, lib), [os.path.join(OBJ, s + ".o") for s in srcs]
        out.append(dst)
        if not os.path.exists(dst) or os.path.getmtime(dst) < max(os.path.getmtime(o) for o in objs):
            _finish(lib, _run([_nvcc(), *ARCH, "-shared", *objs, "-o", dst + ".tmp"], verbose), verbose)
            os.replace(dst + ".tmp", dst)
    return out


if __name__ == "__main__":
    force = "--force" in sys.argv
    extra = ["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else []
    for p in build(force=force or bool(extra), verbose=True, extra=extra):
        print("built", p)
