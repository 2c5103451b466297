"""Build libdcp.so in-tree: nvcc for sm_103a, one object per .cu file compiled in parallel; beside
it the binding's optional helper _tensor_views.so (g++, against the installed torch)."""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
OUT = os.path.join(PKG, "libdcp.so")
VIEWS_SRC = os.path.join(CSRC, "tensor_views.cpp")
VIEWS = os.path.join(PKG, "_tensor_views.so")
BUILD_DIR = os.path.join(os.path.dirname(PKG), "_build")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps() -> list[str]:
    hdr = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    inc = os.path.join(os.path.dirname(PKG), "include")
    hdr += [os.path.join(inc, f) for f in os.listdir(inc)]
    return sources() + hdr + [os.path.abspath(__file__)]


def up_to_date() -> bool:
    if not os.path.exists(OUT):
        return False
    t = os.path.getmtime(OUT)
    return all(os.path.getmtime(p) <= t for p in _deps())


def build_views(force: bool = False) -> None:
    """The binding's helper; without it (no compiler for it, no headers) the binding works all the same."""
    own_inc = os.path.join(os.path.dirname(PKG), "include")
    newest = max(os.path.getmtime(p) for p in (VIEWS_SRC, os.path.join(own_inc, "dcp.h"), os.path.abspath(__file__)))
    import torch
    built_for = f"{torch.__version__} {sys.version_info[:2]}\n"
    stamp = os.path.join(BUILD_DIR, "tensor_views.txt")
    old = open(stamp).read() if os.path.exists(stamp) else None
    if not force and os.path.exists(VIEWS) and os.path.getmtime(VIEWS) >= newest and old == built_for:
        return
    root = os.path.dirname(torch.__file__)
    lib = os.path.join(root, "lib")
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], own_inc]
    tmp = VIEWS + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "g++", "-O1", "-std=c++17", "-fPIC", "-shared", *[f"-I{p}" for p in inc], VIEWS_SRC, "-o", tmp,
           f"-L{lib}", f"-Wl,-rpath,{lib}", "-ltorch_python", "-ltorch_cpu", "-lc10",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        error = r.stderr if r.returncode else ""
    except OSError as e:
        error = str(e)
    if error:
        print(f"_tensor_views.so not built (the binding goes without):\n{error[-2000:]}", file=sys.stderr)
        if os.path.exists(VIEWS):
            os.remove(VIEWS)
        return
    os.replace(tmp, VIEWS)
    os.makedirs(BUILD_DIR, exist_ok=True)
    with open(stamp, "w") as f:
        f.write(built_for)


def build(force: bool = False, verbose: bool = False) -> str:
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        views = ex.submit(build_views, force)
        out = _build_library(force, verbose)
        views.result()
    return out


def _build_library(force: bool, verbose: bool) -> str:
    if not force and up_to_date():
        return OUT
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    objs = []

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and r.stderr.strip():
            print(r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, sources()))
    tmp = OUT + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, OUT)
    return OUT


if __name__ == "__main__":
    print(build(force=True, verbose=True))
